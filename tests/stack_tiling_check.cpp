// Prints how the stages of stacks are divided among workgroups: for every line "count rows cols" of
// the input one line for each stage, "stage tile kind", kind being whole (a workgroup a tile), more or
// fewer (workgroups that share K steps, more or fewer of them than tiles).  Built with g++ by
// tests/test_stack_scale.py from the host source that makes the choice.
#include <cstdio>
#include <cstdlib>

#include "muon_stack.cpp"

namespace muon {

int report(const Status&) { std::abort(); }
int report_exception(const char*) { std::abort(); }
int check_no_alias(const Range*, int, Status*) { std::abort(); }
int check_scalar(float, const char*, Status*) { std::abort(); }
hipError_t launch_stack(const muon_stack_t&, const StackPlan&, float, void*, size_t, hipStream_t) { std::abort(); }
bool stack_is_whole(const StackShape& s) { return stack_whole_lds(s) <= kStackWholeLds; }

}  // namespace muon

extern "C" const char* hipGetErrorString(hipError_t) { return ""; }

int main() {
    long long count, rows, cols;
    while (std::scanf("%lld %lld %lld", &count, &rows, &cols) == 3) {
        const muon::StackShape s = muon::stack_shape(rows, cols);
        if (s.r <= 128) continue;
        for (int stage : {muon::kStageA, muon::kStageB, muon::kStageX}) {
            const muon::StackTiling t = muon::stack_tiling(stage, s, count);
            std::printf("%c %d %s\n", "ABX"[stage], t.tile,
                        t.workers == t.tiles ? "whole" : t.workers > t.tiles ? "more" : "fewer");
        }
    }
    return 0;
}
