// Shared by the kernels of the paged 8-bit key/value cache: its layout, the
// step descriptor, and how a kernel finds the sequence that a work item is of.
#pragma once

#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace nvq {

// codes [P, H, block, D] (one byte a value), scales fp32 [P, H], for K and V.
struct KvCache {
    uint8_t* k_codes;
    float* k_scales;
    uint8_t* v_codes;
    float* v_scales;
    int64_t P;
    int H, block, D;
    int mode;  // NV_KV_INT8 or NV_KV_E4M3
};

// Sequence s: lens[s] tokens, the last starts[s + 1] - starts[s] of them are
// rows starts[s] .. starts[s + 1] of this step; its j-th block of tokens is
// page pages[s * max_pages + j]. All device memory, so nothing here is trusted:
// seq_span and page_of clamp every value before it is used as an index.
struct KvSteps {
    const int32_t* pages;
    const int32_t* starts;
    const int32_t* lens;
    int64_t max_pages;
    int S;
    int64_t rows;  // T
    uint32_t* flags;  // may be null
};

// Places are 32-bit; the rest is room for a chunk's or tile's end behind them.
constexpr int kMaxLen = 0x7FFF0000;

struct SeqSpan {
    int64_t row0;  // first row of the step
    int n;         // rows
    int len;       // tokens, this step's included (at most max_pages * block)
    int first;     // place of the first row in the sequence: len - n, negative if n > len
};

__device__ __forceinline__ int64_t clamped_start(const KvSteps& st, int s) {
    const int64_t v = __ldg(st.starts + s);
    return v < 0 ? 0 : v > st.rows ? st.rows : v;
}

__device__ __forceinline__ SeqSpan seq_span(const KvSteps& st, int s, int block) {
    SeqSpan r;
    const int32_t a0 = __ldg(st.starts + s), a1 = __ldg(st.starts + s + 1), l0 = __ldg(st.lens + s);
    r.row0 = clamped_start(st, s);
    const int64_t r1 = clamped_start(st, s + 1);
    r.n = r1 > r.row0 ? static_cast<int>(r1 - r.row0) : 0;
    const int64_t room = st.max_pages * block;
    const int64_t cap = room < kMaxLen ? room : kMaxLen;
    r.len = l0 < 0 ? 0 : l0 > cap ? static_cast<int>(cap) : l0;
    r.first = r.len - r.n;
    if (st.flags && (a0 < 0 || a1 < a0 || a1 > st.rows || l0 < 0 || l0 > cap || r.n > r.len))
        atomicOr(st.flags, NV_FLAG_BAD_LENGTH);
    return r;
}

// Page of block j of sequence s, or -1 (flagged) if the table names none.
__device__ __forceinline__ int page_of(const KvSteps& st, const KvCache& c, int s, int j) {
    const int32_t p = __ldg(st.pages + static_cast<int64_t>(s) * st.max_pages + j);
    if (p >= 0 && p < c.P) return p;
    if (st.flags) atomicOr(st.flags, NV_FLAG_PAGE_OUT_OF_RANGE);
    return -1;
}

// Work items are laid out sequence by sequence without a table: sequence s
// owns the items from floor(starts[s] * mul / per) + s * extra on, which is at
// least as many as its rows can need. Bounds the items of all sequences:
__host__ __device__ inline int64_t kv_items(int64_t rows, int S, int64_t mul, int64_t per, int extra) {
    return rows * mul / per + static_cast<int64_t>(S) * extra;
}
__device__ __forceinline__ int64_t kv_first_item(const KvSteps& st, int s, int64_t mul, int64_t per, int extra) {
    return clamped_start(st, s) * mul / per + static_cast<int64_t>(s) * extra;
}
// The last sequence whose items start at or before `item`, by one warp: the starts
// ascend, so it is their count. Up to kProbe starts a lane are read at once (256
// sequences in one round trip to memory); more sequences are narrowed first,
// 32 probes a step. The lengths' lines are touched beside them for seq_span.
constexpr int kProbe = 8;
__device__ __forceinline__ int kv_find_seq(const KvSteps& st, int64_t item, int64_t mul, int64_t per, int extra) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = st.S;
    while (hi - lo > 32 * kProbe) {
        const int step = (hi - lo + 31) / 32;
        const int p = lo + lane * step;
        const bool at_or_before = p < hi && kv_first_item(st, p, mul, per, extra) <= item;
        const int n = __popc(__ballot_sync(0xffffffffu, at_or_before));
        lo += (n > 0 ? n - 1 : 0) * step;
        hi = hi < lo + step ? hi : lo + step;
    }
    int before = 0;
#pragma unroll
    for (int i = 0; i < kProbe; ++i) {
        const int p = lo + i * 32 + lane;
        if (lo + i * 32 < hi && p < hi) {
            before += kv_first_item(st, p, mul, per, extra) <= item;
            asm volatile("{\n\t.reg .b32 unused;\n\tld.global.nc.b32 unused, [%0];\n\t}" ::"l"(st.lens + p));
        }
    }
    before = __reduce_add_sync(0xffffffffu, before);
    return before > 0 ? lo + before - 1 : lo;
}

constexpr float kInt8Max = 127.f;
constexpr float kE4m3Max = 448.f;

// One code as a float (exact).
template <int MODE>
__device__ __forceinline__ float code_value(uint32_t byte) {
    if constexpr (MODE == NV_KV_INT8) {
        return static_cast<float>(static_cast<int8_t>(byte));
    } else {
        __nv_fp8_e4m3 v;
        v.__x = static_cast<__nv_fp8_storage_t>(byte);
        return static_cast<float>(v);
    }
}

cudaError_t launch_kv_quantize(const void* k, const void* v, int64_t k_stride, int64_t v_stride, int dt,
                               const KvCache& c, const KvSteps& st, cudaStream_t stream);
cudaError_t launch_kv_dequantize(void* k, void* v, int dt, const KvCache& c, const KvSteps& st,
                                 cudaStream_t stream);

// Attention: q [rows, Hq, D] with a row stride, out [rows, Hq, D].
struct KvAttn {
    const void* q;
    int64_t q_stride;
    void* out;
    int dt, Hq;
    float scale;
    int causal;
    int window;  // 0: none
};
// Plain kernel: any head size, fp32 or bf16, one CTA per (row, query head).
cudaError_t launch_kv_attn_simple(const KvAttn& a, const KvCache& c, const KvSteps& st, cudaStream_t stream);

// Kernel for few rows a sequence (bf16, D 64 or 128): sequences are cut into
// chunks that a second kernel joins. `only`: every sequence is its; else it takes those of at
// most 16 flattened rows (token, head of the group) and leaves the others. `beside`: it is launched behind the
// kernel for many rows, nothing of whose it reads, and begins when that one's last CTAs have.
struct KvDecodeSizes {
    int64_t rows, S, max_pages;
    int Hq, H, block, D;
    bool only;
    int64_t G, most_rows;  // heads of a group; most flattened rows a sequence has
};
// Bytes of the partial outputs and log-sums of `rows` rows, at most 2^50: no workspace holds those, so
// that such a call is refused, and the sizes of two kernels add up without wrapping around.
inline size_t kv_part_bytes(int64_t rows, int64_t parts, int D) {
    constexpr size_t kMost = static_cast<size_t>(1) << 50;
    const size_t row = static_cast<size_t>(parts) * (D + 1) * sizeof(float);
    return static_cast<size_t>(rows) > kMost / row ? kMost : static_cast<size_t>(rows) * row;
}
struct KvDecodePlan {
    int target, max_chunks, tile_rows, row_limit;
    int64_t part_rows;
    size_t bytes(int D) const { return max_chunks > 1 ? kv_part_bytes(part_rows, max_chunks, D) : 0; }
};
KvDecodePlan kv_decode_plan(const KvDecodeSizes& z, int num_sms);
cudaError_t launch_kv_attn_decode(const KvAttn& a, const KvCache& c, const KvSteps& st, const KvDecodePlan& plan,
                                  void* workspace, bool beside, cudaStream_t stream, int num_sms);
unsigned int kv_attn_decode_error_take();

// Tensor-core kernel for many rows a sequence (bf16, D 64 or 128); sequences of at
// most row_min flattened rows are left to the other. A second launch joins the parts that tokens were cut into.
struct KvPrefillSizes {
    int64_t rows, S, max_pages;
    int Hq, H, block, D;
};
struct KvPrefillPlan {
    int64_t items;
    int splits;
    size_t bytes(int64_t rows, int Hq, int D) const { return splits > 1 ? kv_part_bytes(rows * Hq, splits, D) : 0; }
};
KvPrefillPlan kv_prefill_plan(const KvPrefillSizes& z, int num_sms);
cudaError_t launch_kv_attn_prefill(const KvAttn& a, const KvCache& c, const KvSteps& st, const KvPrefillPlan& plan,
                                   int row_min, void* workspace, cudaStream_t stream);
cudaError_t launch_kv_attn_prefill_join(const KvAttn& a, const KvCache& c, const KvSteps& st, const KvPrefillPlan& plan,
                                        int row_min, void* workspace, cudaStream_t stream);
unsigned int kv_attn_prefill_error_take();

}  // namespace nvq
