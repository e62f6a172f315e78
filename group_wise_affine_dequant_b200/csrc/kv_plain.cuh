// One query row of the attention over the paged 8-bit cache, plainly, by 128 threads:
//   z_j = scale * k_scale[page of j] * (q . k_code_j),  p = softmax(z),
//   out = sum_j p_j * v_scale[page of j] * v_code_j
// over the row's visible tokens, 128 at a time with a running maximum and sum. A
// thread computes one token's score, then owns values d, d + 128 of the output.
// Everything is fp32, and stays in its range wherever scores and values do: queries are taken
// times a power of two that the scores get back, and what is kept of the output is its mean so far, no sum.
#pragma once

#include "kv.cuh"

namespace nvq {

constexpr int kPlainThreads = 128;

template <int D>  // the most values a head has
struct PlainScratch {
    int64_t at[kPlainThreads];  // where token j's values start in v_codes
    float w[kPlainThreads];     // p_j * v_scale / 128
    float q[D];
    float red[2][kPlainThreads / 32];
};

struct PlainRow {
    float out[2];  // values tid and tid + 128
    float m, l;    // the largest score and the sum of e^(z - m); -infinity and 0 where nothing is seen
};

// Row t of the step, of sequence s, against the tokens it sees in [from, to). `sync` is a
// barrier of the 128 threads, of which this one is `tid`; all of them get the same m and l.
template <int DT, int MODE, int MAXD, class Sync>
__device__ __forceinline__ PlainRow plain_row(const KvAttn& a, const KvCache& c, const KvSteps& st, int s, const SeqSpan& span,
                                              int64_t t, int hq, int from, int to, int tid, PlainScratch<MAXD>& x,
                                              const Sync& sync) {
    const int lane = tid & 31, warp = tid >> 5, h = hq / (a.Hq / c.H);
    const int64_t pos = span.first + (t - span.row0);
    int hi = a.causal ? (pos + 1 < span.len ? static_cast<int>(pos + 1) : span.len) : span.len;
    int lo = a.window > 0 && pos + 1 > a.window ? static_cast<int>(pos + 1 - a.window) : 0;
    hi = hi < to ? hi : to;
    lo = lo > from ? lo : from;
    const int64_t q0 = t * a.q_stride + static_cast<int64_t>(hq) * c.D;
    float raw[2];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int d = tid + i * kPlainThreads;
        raw[i] = d < c.D ? load_elem<DT>(a.q, q0 + d) : 0.f;
        top = max(top, __float_as_uint(raw[i]) & 0x7FFFFFFFu);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) x.red[0][warp] = __uint_as_float(top);
    sync();
#pragma unroll
    for (int i = 0; i < kPlainThreads / 32; ++i) top = max(top, __float_as_uint(x.red[0][i]));
    if (top >= 0x7F800000u) {  // not finite: else scores of -infinity alone would pass for nothing seen
        sync();                // before the scratch is another row's
        return PlainRow{{NAN, NAN}, 0.f, NAN};
    }
    uint32_t ex = top >> 23;
    // 2^7 and more: up to 2^100, so that what the scores get back times a large key scale stays finite; below
    // 2^-119: both powers of two stay normal numbers
    ex = ex < 8u ? 8u : ex <= 133u ? ex : ex <= 233u ? 133u : ex - 100u;
    const float down = __uint_as_float((254u - ex) << 23), zc = a.scale * __uint_as_float(ex << 23);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (tid + i * kPlainThreads < c.D) x.q[tid + i * kPlainThreads] = raw[i] * down;
    sync();

    PlainRow r{{0.f, 0.f}, -INFINITY, 0.f};
    for (int j0 = lo; j0 < hi; j0 += kPlainThreads) {
        const int j = j0 + tid;
        float z = -INFINITY, vs = 0.f;
        int64_t row = 0;
        if (j < hi) {
            const int page = page_of(st, c, s, j / c.block);
            if (page >= 0) {
                const int64_t ph = static_cast<int64_t>(page) * c.H + h;
                row = (ph * c.block + j % c.block) * c.D;
                vs = __ldg(c.v_scales + ph);
                const uint4* k = reinterpret_cast<const uint4*>(c.k_codes + row);
                float dot = 0.f;
                for (int i = 0; i < c.D / 16; ++i) {
                    const uint4 u = __ldg(k + i);
                    const uint32_t y[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        dot = fmaf(x.q[16 * i + e], code_value<MODE>(y[e / 4] >> (8 * (e & 3)) & 255u), dot);
                }
                z = dot * (zc * __ldg(c.k_scales + ph));
            }
        }
        float most = z;
#pragma unroll
        for (int o = 16; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
        if (lane == 0) x.red[0][warp] = most;
        sync();
        most = fmaxf(fmaxf(x.red[0][0], x.red[0][1]), fmaxf(x.red[0][2], x.red[0][3]));
        const float m2 = fmaxf(r.m, most);
        const float base = m2 == -INFINITY ? 0.f : m2;  // nothing visible yet: every p is 0
        const float p = expf(z - base);
        float part = p;
#pragma unroll
        for (int o = 16; o; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
        if (lane == 0) x.red[1][warp] = part;
        x.w[tid] = p * vs * (1.f / kPlainThreads);
        x.at[tid] = row;
        sync();
        const float held = r.l * expf(r.m - base);
        r.l = held + ((x.red[1][0] + x.red[1][1]) + (x.red[1][2] + x.red[1][3]));
        r.m = m2;
        float acc[2] = {0.f, 0.f};  // of 128 tokens, over 128: no larger than the largest value
        const int count = hi - j0 < kPlainThreads ? hi - j0 : kPlainThreads;
        for (int i = 0; i < count; ++i) {
            const float wi = x.w[i];
            if (wi == 0.f) continue;
            if (tid < c.D) acc[0] = fmaf(wi, code_value<MODE>(__ldg(c.v_codes + x.at[i] + tid)), acc[0]);
            if (tid + kPlainThreads < c.D)
                acc[1] = fmaf(wi, code_value<MODE>(__ldg(c.v_codes + x.at[i] + tid + kPlainThreads)), acc[1]);
        }
        const float inv = r.l > 0.f || r.l != r.l ? 1.f / r.l : 0.f;  // nothing visible: zeros
#pragma unroll
        for (int i = 0; i < 2; ++i) r.out[i] = fmaf(acc[i], kPlainThreads * inv, r.out[i] * (held * inv));
        sync();
    }
    return r;
}

}  // namespace nvq
