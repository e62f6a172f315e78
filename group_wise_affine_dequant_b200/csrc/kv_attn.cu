// Attention over the paged 8-bit cache: the plain kernel, which takes every
// head size and type, one CTA per (row, query head). It reads the cache once per query
// head (a group of heads shares it through the L2) and is bound by its fp32 arithmetic.
#include <cstdint>

#include "kv_plain.cuh"
#include "tma.cuh"

namespace nvq {
namespace {

template <int DT, int MODE>
__global__ void __launch_bounds__(kPlainThreads) kv_attn_simple_kernel(const __grid_constant__ KvAttn a,
                                                                       const __grid_constant__ KvCache c,
                                                                       const __grid_constant__ KvSteps st) {
    __shared__ PlainScratch<256> scratch;
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x;
    const int64_t t = blockIdx.x / a.Hq;
    const int hq = static_cast<int>(blockIdx.x - t * a.Hq);
    const int s = kv_find_seq(st, t, 1, 1, 0);
    const SeqSpan span = seq_span(st, s, c.block);
    if (t < span.row0 || t >= span.row0 + span.n) return;  // no sequence's row: left as it was
    const PlainRow r = plain_row<DT, MODE>(a, c, st, s, span, t, hq, 0, span.len, tid, scratch, [] { __syncthreads(); });
    const int64_t o = (t * a.Hq + hq) * c.D;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (tid + i * kPlainThreads < c.D) store_elem<DT>(a.out, o + tid + i * kPlainThreads, r.out[i]);
}

template <int DT, int MODE>
cudaError_t launch(const KvAttn& a, const KvCache& c, const KvSteps& st, cudaStream_t stream) {
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(st.rows * a.Hq), 1, 1);
    cfg.blockDim = dim3(kPlainThreads, 1, 1);
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
