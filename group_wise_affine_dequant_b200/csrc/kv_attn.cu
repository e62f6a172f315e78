// Attention over the paged 8-bit cache: the plain kernel, which takes every
// head size and type. One CTA per (row, query head):
//   z_j = scale * k_scale[page of j] * (q . k_code_j),  p = softmax(z),
//   out = sum_j p_j * v_scale[page of j] * v_code_j
// over the row's visible tokens, 128 at a time with a running maximum and sum.
// A thread computes one token's score, then owns values d, d + 128 of the
// output. Everything is fp32. It reads the cache once per query head (a group
// of heads shares it through the L2) and is bound by its fp32 arithmetic.
#include <cstdint>

#include "kv.cuh"
#include "tma.cuh"

namespace nvq {
namespace {

constexpr int kThreads = 128;

template <int DT, int MODE>
__global__ void __launch_bounds__(kThreads) kv_attn_simple_kernel(const __grid_constant__ KvAttn a,
                                                                  const __grid_constant__ KvCache c,
                                                                  const __grid_constant__ KvSteps st) {
    __shared__ float q[256];
    __shared__ float w[kThreads];         // p_j * v_scale
    __shared__ int64_t at[kThreads];      // where token j's values start in v_codes
    __shared__ float red[2][kThreads / 32];
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t t = blockIdx.x / a.Hq;
    const int hq = static_cast<int>(blockIdx.x - t * a.Hq), h = hq / (a.Hq / c.H);
    const int s = kv_find_seq(st, t, 1, 1, 0);
    const SeqSpan span = seq_span(st, s, c.block);
    if (t < span.row0 || t >= span.row0 + span.n) return;  // no sequence's row: left as it was
    const int64_t pos = span.first + (t - span.row0);
    const int hi = a.causal ? (pos + 1 < span.len ? static_cast<int>(pos + 1) : span.len) : span.len;
    const int lo = a.window > 0 && pos + 1 > a.window ? static_cast<int>(pos + 1 - a.window) : 0;
    for (int d = tid; d < c.D; d += kThreads)
        q[d] = load_elem<DT>(a.q, t * a.q_stride + static_cast<int64_t>(hq) * c.D + d) * a.scale;
    __syncthreads();

    float m = -INFINITY, l = 0.f, acc[2] = {0.f, 0.f};
    for (int j0 = lo; j0 < hi; j0 += kThreads) {
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
                    const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        dot = fmaf(q[16 * i + e], code_value<MODE>(x[e / 4] >> (8 * (e & 3)) & 255u), dot);
                }
                z = dot * __ldg(c.k_scales + ph);
            }
        }
        float most = z;
#pragma unroll
        for (int o = 16; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
        if (lane == 0) red[0][warp] = most;
        __syncthreads();
        most = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
        const float m2 = fmaxf(m, most);
        const float base = m2 == -INFINITY ? 0.f : m2;  // nothing visible yet: every p is 0
        const float p = expf(z - base);
        float part = p;
#pragma unroll
        for (int o = 16; o; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
        if (lane == 0) red[1][warp] = part;
        w[tid] = p * vs;
        at[tid] = row;
        __syncthreads();
        const float grow = expf(m - base);
        l = l * grow + ((red[1][0] + red[1][1]) + (red[1][2] + red[1][3]));
        acc[0] *= grow;
        acc[1] *= grow;
        m = m2;
        const int count = hi - j0 < kThreads ? hi - j0 : kThreads;
        for (int i = 0; i < count; ++i) {
            const float wi = w[i];
            if (wi == 0.f) continue;
            if (tid < c.D) acc[0] = fmaf(wi, code_value<MODE>(__ldg(c.v_codes + at[i] + tid)), acc[0]);
            if (tid + kThreads < c.D)
                acc[1] = fmaf(wi, code_value<MODE>(__ldg(c.v_codes + at[i] + tid + kThreads)), acc[1]);
        }
        __syncthreads();
    }
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;  // nothing visible: zeros
    const int64_t o = (t * a.Hq + hq) * c.D;
    if (tid < c.D) store_elem<DT>(a.out, o + tid, acc[0] * inv);
    if (tid + kThreads < c.D) store_elem<DT>(a.out, o + tid + kThreads, acc[1] * inv);
}

template <int DT, int MODE>
cudaError_t launch(const KvAttn& a, const KvCache& c, const KvSteps& st, cudaStream_t stream) {
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(st.rows * a.Hq), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = stream;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_attn_simple_kernel<DT, MODE>, a, c, st);
}

}  // namespace

cudaError_t launch_kv_attn_simple(const KvAttn& a, const KvCache& c, const KvSteps& st, cudaStream_t stream) {
    if (a.dt == NV_F32)
        return c.mode == NV_KV_INT8 ? launch<NV_F32, NV_KV_INT8>(a, c, st, stream)
                                    : launch<NV_F32, NV_KV_E4M3>(a, c, st, stream);
    return c.mode == NV_KV_INT8 ? launch<NV_BF16, NV_KV_INT8>(a, c, st, stream)
                                : launch<NV_BF16, NV_KV_E4M3>(a, c, st, stream);
}

}  // namespace nvq
