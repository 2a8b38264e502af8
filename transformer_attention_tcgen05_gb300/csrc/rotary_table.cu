// The table of rotary positions (host): theta_i / (2 pi) to the nearest 2^-64 of a turn.
//
// A position t turns by t theta_i, so an error of the table grows with t: made from
// 53-bit numbers it would be 2^-24 of a turn at position 2^31.  Numbers here are sums of
// two doubles (some 100 bits): a sum's or a product's rounding error is a double itself,
// found by the additions of Knuth and by a fused multiply-add.  exp is its power series
// of a reduced argument, squared; log a Newton step on exp; pi and ln 2 are series too.
#include <math.h>
#include <stdint.h>

#include "kernels.h"

namespace attn {
namespace {

struct Wide {
    double hi, lo;
};

// A product that the compiler may not contract with an addition behind it.
double product(double a, double b) {
    volatile double p = a * b;
    return p;
}
Wide exact_sum(double a, double b) {
    const double s = a + b, t = s - a;
    return Wide{s, (a - (s - t)) + (b - t)};
}
Wide exact_product(double a, double b) {
    const double p = product(a, b);
    return Wide{p, fma(a, b, -p)};
}
Wide add(Wide a, Wide b) {
    const Wide s = exact_sum(a.hi, b.hi), t = exact_sum(a.lo, b.lo);
    const Wide u = exact_sum(s.hi, s.lo + t.hi);
    return exact_sum(u.hi, u.lo + t.lo);
}
Wide mul(Wide a, Wide b) {
    const Wide p = exact_product(a.hi, b.hi);
    return exact_sum(p.hi, p.lo + (product(a.hi, b.lo) + product(a.lo, b.hi)));
}
Wide wide(double x) { return Wide{x, 0.0}; }
Wide neg(Wide a) { return Wide{-a.hi, -a.lo}; }
Wide scaled(Wide a, int e) { return Wide{ldexp(a.hi, e), ldexp(a.lo, e)}; }
Wide div(Wide a, Wide b) {
    Wide q = wide(0.0);
    for (int i = 0; i < 3; ++i) {
        const Wide d = wide(a.hi / b.hi);
        q = add(q, d);
        a = add(a, neg(mul(d, b)));
    }
    return q;
}

// sum over k of sign^k / ((2 k + 1) n^(2 k + 1)): the inverse tangent of 1 / n
// (sign -1), or its hyperbolic one (1).
Wide inverse_tangent(int n, int sign) {
    Wide power = div(wide(1.0), wide(n)), sum = power;
    for (int k = 1; k < 40; ++k) {
        power = div(power, wide(double(sign) * n * n));
        sum = add(sum, div(power, wide(2 * k + 1)));
    }
    return sum;
}

struct Constants {
    // ln 2 = 2 artanh(1/3); pi = 16 arctan(1/5) - 4 arctan(1/239) (Machin)
    Wide ln2 = scaled(inverse_tangent(3, 1), 1);
    Wide two_pi = scaled(add(scaled(inverse_tangent(5, -1), 2), neg(inverse_tangent(239, -1))), 3);
};

Wide exponential(Wide x, const Constants &c) {
    if (!(fabs(x.hi) < 1e4)) return wide(x.hi > 0 ? INFINITY : 0.0);
    const double k = nearbyint(x.hi / c.ln2.hi);
    const Wide r = scaled(add(x, neg(mul(wide(k), c.ln2))), -9);   // at most ln 2 / 2^10
    Wide term = wide(1.0), sum = term;
    for (int i = 1; i < 12; ++i) {
        term = div(mul(term, r), wide(i));
        sum = add(sum, term);
    }
    for (int i = 0; i < 9; ++i) sum = mul(sum, sum);
    return scaled(sum, int(k));
}

// Of a positive finite number.
Wide logarithm(double x, const Constants &c) {
    int e;
    const double m = frexp(x, &e);
    Wide y = wide(log(m));
    for (int i = 0; i < 2; ++i) y = add(y, add(mul(wide(m), exponential(neg(y), c)), wide(-1.0)));
    return add(y, mul(wide(e), c.ln2));
}

}  // namespace

attn_status_t rope_frequencies(uint64_t *freq, int rot, double theta, attn_rope_scaling_t scaling, double factor,
                               double original_len, double alpha, double beta) {
    static const Constants c;
    Wide base = logarithm(theta, c);
    if (scaling == ATTN_ROPE_NTK)
        base = add(base, div(mul(logarithm(factor, c), wide(rot)), wide(rot - 2)));
    // turns per position, unscaled, of a pair and of the next one for each
    Wide turns = div(wide(1.0), c.two_pi);
    const Wide ratio = exponential(div(mul(base, wide(-2.0)), wide(rot)), c);
    for (int i = 0; i < rot / 2; ++i, turns = mul(turns, ratio)) {
        Wide f = turns;
        if (scaling == ATTN_ROPE_LINEAR) {
            f = div(f, wide(factor));
        } else if (scaling == ATTN_ROPE_BY_PARTS) {
            const Wide above = add(mul(wide(original_len), f), wide(-alpha));
            Wide share = div(above, exact_sum(beta, -alpha));
            if (!(share.hi > 0)) share = wide(0.0);
            if (share.hi >= 1) share = wide(1.0);
            f = add(div(mul(add(wide(1.0), neg(share)), f), wide(factor)), mul(share, f));
        }
        const Wide t = scaled(f, 64);
        // half a turn per position or more, or no number
        if (!(f.hi < 0.5) || !isfinite(t.lo)) return ATTN_ERR_INVALID_ARG;
        const double whole = floor(t.hi);
        freq[i] = uint64_t(whole) + uint64_t(int64_t(floor((t.hi - whole) + t.lo + 0.5)));
    }
    return ATTN_OK;
}

}  // namespace attn
