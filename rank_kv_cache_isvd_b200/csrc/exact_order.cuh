// The order in which the split and rows kernels visit the rows that a tile of query tokens sees: plain
// arithmetic, the same on host and device.
//
// Token i of a sequence of n rows and ql tokens sits at p = n - ql + i and sees the rows j <= p with
// j < sinks or j > p - window. Tokens i0 .. i1 - 1 together see the sinks and the rows from the first
// token's window on. Where the window does not reach the sinks, the order leaves out the gap: c < skp are
// the sinks (sk of them, filled up to a multiple of a warp's rows), then the rows from lo on, up to C.
// Filling by a warp's rows gives every warp's step below C a row, and none of them both parts.
#pragma once

#ifdef __CUDACC__
#define EX_HD __host__ __device__ __forceinline__
#else
#define EX_HD inline
#endif

namespace iskv {

// Rows per warp and step.
EX_HD constexpr int ex_warp_rows(bool f32_rows) { return f32_rows ? 16 : 32; }

struct ExactOrder {
    int C, sk, skp, lo;
};

EX_HD int ex_fill(int sk, int wr) { return (sk + wr - 1) & ~(wr - 1); }

EX_HD ExactOrder ex_order(int n, int ql, int i0, int i1, int window, int sinks, int wr) {
    const int p = n - ql + i0 - window + 1, hi = n - ql + i1 > 0 ? n - ql + i1 : 0;
    const int sk = sinks < hi ? sinks : hi, lo = p > 0 ? p : 0;
    ExactOrder o = {hi, 0, 0, 0};
    if (lo > sk) {
        o.sk = sk;
        o.skp = ex_fill(sk, wr);
        o.lo = lo;
        o.C = o.skp + hi - lo;
    }
    return o;
}

// Row at place c of the order (c of the sinks' filling: rows behind them, which nobody sees).
EX_HD int ex_row(const ExactOrder &o, int c) { return c < o.skp ? c : c - o.skp + o.lo; }

// Of the wr places from c on (a multiple of wr): how many, from the first, have a row behind them.
EX_HD int ex_seen(const ExactOrder &o, int c, int wr) {
    const int left = (c < o.skp ? o.sk : o.C) - c;
    return left < 0 ? 0 : left < wr ? left : wr;
}

// C at most, of tpt tokens of a sequence of n rows.
EX_HD int ex_most_rows(int window, int sinks, int tpt, int n, int wr) {
    const long long most = (long long)ex_fill(sinks, wr) + window + tpt - 1;
    const int all = window >= n ? n : n + wr - 1;
    return most < all ? (int)most : all;
}

}  // namespace iskv
