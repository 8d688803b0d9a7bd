// Host-only checks of the exponents with which the iterates of a stack are stored, and of the
// factors that follow from them.  Built with g++ by tests/test_stack_scale.py; prints "ok".
//
// A 1 x 1 matrix runs through the same exponents and factors as any other, in float32: every
// stored number has to stay within float16's range and every result within float32 roundings of
// the iteration in float64, for first iterates of every size.
#include <cstdio>
#include <cstdlib>
#include <initializer_list>
#include <vector>

#include "stack_internal.h"

using namespace muon;

namespace {

int g_checked = 0;

void fail(const char* what, double x, size_t step, double got, double want) {
    std::printf("%s: x = %g, step %zu: %g, expected %g\n", what, x, step, got, want);
    std::exit(1);
}

// Steps from a first iterate of x, its bound `top` (>= x), times `scale`.
void run(const std::vector<StackStep>& steps, float x, float top, float scale) {
    const double x0 = x;
    double want = x;
    int sx = stack_exponent(top, kStackLeastX);
    if (sx > 127) fail("exponent of the first iterate", x0, 0, sx, 127);
    float held = x * stack_scaled(1.f, sx);
    for (size_t t = 0; t < steps.size(); ++t) {
        const StackStep& k = steps[t];
        const StackScale s = stack_scale(k, top);
        if (s.sx != sx) fail("exponent of a later iterate", x0, t, s.sx, sx);
        const bool last = t + 1 == steps.size();
        const int next = stack_exponent(top, kStackLeastX);
        const StackFactors b = stack_b_factors(k, s), f = stack_x_factors(k, s, next, last, scale);
        for (float v : {stack_a_factor(s), b.own, b.down, f.own, f.down, f.after})
            if (!std::isfinite(v)) fail("a factor", x0, t, v, 0);
        const float gram = held * held * stack_a_factor(s);
        const float poly = gram * b.own + gram * gram * b.down;
        for (float v : {held, gram, poly})
            if (!(std::fabs(v) <= 65504.f)) fail("a stored number", x0, t, v, 65504);
        held = (f.own * held + f.down * (held * poly)) * f.after;
        want = k.a * want + k.b * want * want * want + k.c * want * want * want * want * want;
        // relative to the bound of the results; float32 numbers below 2^-126 lose digits
        double got = last ? held : std::ldexp(double(held), -next);
        const double size = last ? double(scale) * want : want;
        const double bound = double(top) * (last ? std::fabs(double(scale)) : 1.);
        if (!(std::fabs(got - size) <= 1e-5 * bound + std::ldexp(1., -140))) fail("a result", x0, t, got, size);
        sx = next;
        ++g_checked;
    }
}

// The bound of a step's results against the largest of them on a fine grid.
void bound(const StackStep& k, float top) {
    double most = 0;
    for (int i = 1; i <= 4000; ++i) {
        const double x = double(top) * i / 4000;
        most = std::fmax(most, std::fabs(x * (k.a + x * x * (k.b + x * x * double(k.c)))));
    }
    const double got = stack_largest(k, top);
    if (!(got >= most * (1 - 1e-5) - 1e-44) || !(got <= most * (1 + 1e-4) + 1e-44)) fail("a bound", top, 0, got, most);
    ++g_checked;
}

}  // namespace

int main() {
    for (const StackStep& k : std::initializer_list<StackStep>{
             {3.4445f, -4.7750f, 2.0315f}, {8.f, -22.f, 15.f}, {30.f, -29.f, 0.f}, {1.f, 0.f, 0.f}, {0.f, 1.f, 0.f},
             {0.f, 0.f, -1.f}, {0.f, -2.f, 1.f}, {3.f, -3.f, 1e-8f}, {3.f, -3.f, -1e-8f}, {3.f, -3.f, 1e-3f},
             {1e-7f, -3.f, 3.f}, {-1e-7f, 3.f, -3.f}, {5.f, -20.f, 16.f}, {-5.f, 20.f, -16.f}, {1.f, -1.f, 1e-20f}})
        // the same polynomial on other intervals, and of other sizes
        for (float top : {1.001f, 1e-3f, 1e-9f, 4e-10f, 300.f})
            for (float size : {1.f, 1e-25f, 1e-33f, 1e4f}) {
                const double t = top, s = size;
                const StackStep scaled{float(k.a * s), float(k.b * s / (t * t)), float(k.c * s / (t * t * t * t))};
                if (std::isfinite(scaled.a) && std::isfinite(scaled.b) && std::isfinite(scaled.c)) bound(scaled, top);
            }
    const StackStep quintic{3.4445f, -4.7750f, 2.0315f};
    const std::vector<std::vector<StackStep>> lists = {
        {quintic},
        {quintic, quintic, quintic, quintic, quintic},
        {{1.875f, -1.25f, 0.375f}, {1.875f, -1.25f, 0.375f}},
        {{0.01f, 0.f, 0.f}, {0.01f, 0.f, 0.f}, {0.01f, 0.f, 0.f}},
        {{0.f, 1.f, 0.f}},
        {{0.f, 0.f, 0.f}, quintic},
        {{1e-30f, 0.f, 0.f}, {1e-30f, 0.f, 0.f}, {1e-30f, 0.f, 0.f}},
        {{1000.f, 0.f, 0.f}, {1e-40f, 0.f, 0.f}, {1.f, 0.f, 0.f}},
        // the iterate shrunk and grown again
        {{1e-5f, 0.f, 0.f}, {1e5f, 0.f, 0.f}, quintic},
        {{1e-9f, 0.f, 0.f}, {5.f, 0.f, 1e38f}, quintic},
        // an end where the polynomial is nearly zero, with a small last coefficient; coefficients for a shrunk iterate
        {{2.598f, -2.598f, 1e-8f}, {1.5f, -0.5f, 0.f}},
        {{1e-9f, 0.f, 0.f}, {5.f, -20e18f, 16e36f}, quintic},
    };
    for (const auto& steps : lists)
        for (float scale : {1.f, -0.2f, 1e-3f, 1e6f})
            // norms of float32 matrices: X = norm / (norm + 1e-7)
            for (int e = -149; e < 128; ++e)
                for (double m : {1., 1.2, 1.999}) {
                    const double norm = double(float(std::ldexp(m, e)));
                    if (norm == 0.) continue;
                    const float top = 1.001f * float(norm / (norm + 1e-7));
                    for (double part : {1., 0.3, 0.}) run(steps, float(part * norm / (norm + 1e-7)), top, scale);
                }
    std::printf("%s\n", g_checked > 100000 ? "ok" : "too few checks");
    return 0;
}
