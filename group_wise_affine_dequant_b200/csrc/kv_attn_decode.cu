// Attention over the paged 8-bit cache for few query rows a sequence (bf16, 64 or
// 128 values a head): the work is reading the cache once.
//
// A row tile is 8 (or 16) query rows of one sequence and key/value head, row =
// (token, query head of the group); an item is a row tile against a chunk of
// the sequence (a multiple of 64 tokens). Items of all sequences are counted
// by every CTA from the lengths (a prefix sum in shared memory), so the grid is
// one wave of resident CTAs and the host needs to know no length.
//
// Per CTA: a producer warp fetches page ids and scales of the next item and
// streams its codes by TMA, 64 tokens of K and V a stage (boxes of
// min(block, 64) tokens, swizzled so that all fragment reads but the 64-wide
// values' are free of bank conflicts). Four consumer warps take 32 tokens of every
// other stage each, with their own running maximum, sum and output. Both products
// are transposed, codes first: S^T = K Q^T and O^T = V^T P^T with mma.m16n8k16, 16
// tokens (or values) by 8 query rows: no half of the instruction is spent on rows
// that a decoding step does not have, and O takes D / 4 registers. Codes become fp16
// (exact) in registers, values transposed byte-wise on the way; the weights' 8 x 8
// blocks turn from accumulators to operands by movmatrix. No barrier between the
// warps inside an item; they join at its end. Items of a sequence that
// takes several write (output, log-sum) to the workspace and a second kernel
// joins them in chunk order, so results do not depend on timing. An item whose value scales are too far apart
// for fp16 weights (2^24) is read row by row in fp32 by the same warps (one such block in
// each of 64 sequences of 8192: 0.14 -> 2.4 ms).
//
// Bound: the code bytes, 2 * D a token and key/value head. What it takes to reach
// them is warps in flight (a warp's step is one long chain): 3 CTAs an SM.
#include <cstdint>

#include "kv_mma.cuh"
#include "kv_plain.cuh"

namespace nvq {
namespace {

constexpr int kTile = 64;        // tokens a stage
constexpr int kConsumers = 4;    // warps
constexpr int kThreads = 32 * (kConsumers + 1);
constexpr int kChunkMax = 1024;  // tokens an item: long enough that joining costs under 2 %
constexpr int kChunkMin = 128;
constexpr int kBlocksMax = kChunkMax / 16 + 1;

constexpr int kCtas = 3;         // resident on an SM

// Even: within an item a stage then belongs to one pair of consumer warps, which frees a filling before it waits
// for the next, so that the parity it waits for cannot be that of the filling before last. From item to
// item a stage may change pairs (an item can have an odd number of them): there the barriers at an item's end, which all
// consumers pass, put one pair's last wait before the other's first.
template <int D>
constexpr int kStages = D == 128 ? 4 : 8;
static_assert(kStages<64> % 2 == 0 && kStages<128> % 2 == 0, "");

struct ItemMeta {
    int64_t row0;       // first row of the sequence in the step
    int h, s;
    int f0, rows;       // the tile's first flattened row (token * G + group head) and its rows
    int first;          // place of the sequence's first row
    int len;
    int t0, t1;         // tokens [t0, t1) of the chunk; t0 a multiple of 64
    int lo_max, hi_min; // tokens in [lo_max, hi_min) are visible to every row of the tile
    int chunk;
    int block0;         // t0 / block
    float vmax;         // largest value scale of the item
    bool direct;        // the sequence's only chunk: the item writes the output, else partials
    bool wide;          // value scales too far apart for fp16 weights: no stages, the rows go one by one
};

// Chunk length for a span of tokens: `target` chunks a sequence where the GPU would be
// short of work, but never so long that one sequence is the tail of the grid; equal parts.
__device__ __forceinline__ int chunk_tokens(int span, int target, int most) {
    const uint32_t s = span, by_most = (s + most - 1) / most;
    const uint32_t n = by_most < static_cast<uint32_t>(target) ? target : by_most;
    const uint32_t c = ((s + n - 1) / n + kTile - 1) / kTile * kTile;
    return static_cast<int>(c < kChunkMin ? kChunkMin : c);
}

struct DecodeArgs {
    KvAttn a;
    KvCache c;
    KvSteps st;
    int target;      // chunks a sequence is cut into (see chunk_tokens)
    int chunk_max;
    int max_chunks;  // partials a row has room for
    int tile_rows;   // 8 or 16
    int lg_block;    // log2 of the cache's block
    int row_limit;   // sequences of more flattened rows are not this kernel's (0: all are)
    bool beside;     // launched on the kernel for many rows, beside whose end it runs
    float* part_o;   // [rows][max_chunks][D]
    float* part_lse; // [rows][max_chunks]
};

// Where a sequence's items come from.
struct SeqWork {
    SeqSpan span;
    int lo;      // first token any row sees, rounded down to 64
    int chunk, chunks, tiles;
};
__device__ __forceinline__ SeqWork seq_work(const DecodeArgs& p, int s) {
    SeqWork w;
    w.span = seq_span(p.st, s, p.c.block);
    const int G = p.a.Hq / p.c.H;
    const int64_t rows = static_cast<int64_t>(w.span.n) * G;
    w.lo = 0;
    if (p.a.window > 0 && w.span.first + 1 > p.a.window) w.lo = (w.span.first + 1 - p.a.window) / kTile * kTile;
    const int span = w.span.len - w.lo;
    w.chunk = chunk_tokens(span > 0 ? span : 1, p.target, p.chunk_max);
    w.chunks = span > 0 ? (span + w.chunk - 1) / w.chunk : 1;  // a row that sees nothing still writes zeros
    w.tiles = static_cast<int>((rows + p.tile_rows - 1) / p.tile_rows);
    if (p.row_limit > 0 && rows > p.row_limit) w.tiles = 0;
    return w;
}
// Partial index of flattened row f of sequence s and head h, chunk 0.
__device__ __forceinline__ int64_t part_row(const DecodeArgs& p, const SeqSpan& span, int s, int h, int f) {
    const int G = p.a.Hq / p.c.H;
    if (p.row_limit > 0) return (static_cast<int64_t>(s) * p.c.H + h) * p.row_limit + f;
    return (span.row0 + f / G) * p.a.Hq + h * G + f % G;
}

// Transpose an 8 x 8 block of 16-bit values: lane 4 g + t holds (g, 2 t), (g, 2 t + 1).
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// The rows of a wide item, one after the other, by the four consumer warps.
template <int MODE, int D>
__device__ __noinline__ void wide_item(const DecodeArgs& p, const ItemMeta& m, PlainScratch<D>& scratch) {
    const int G = p.a.Hq / p.c.H, d = threadIdx.x;
    const SeqSpan span{m.row0, m.len - m.first, m.len, m.first};
    for (int row = 0; row < m.rows; ++row) {
        const int f = m.f0 + row, hq = m.h * G + f % G;
        const int64_t t = m.row0 + f / G;
        const PlainRow r = plain_row<NV_BF16, MODE>(p.a, p.c, p.st, m.s, span, t, hq, m.t0, m.t1, d, scratch,
                                                    [] { asm volatile("bar.sync 1, 128;" ::: "memory"); });
        if (m.direct) {
            if (d < D) static_cast<uint16_t*>(p.a.out)[(t * p.a.Hq + hq) * D + d] = f32_to_bf16_bits(r.out[0]);
        } else {
            const int64_t at = part_row(p, span, m.s, m.h, f) * p.max_chunks + m.chunk;
            if (d < D) p.part_o[at * D + d] = r.out[0];
            // the other items' sums carry 2^kLift, and count no row that is not a number
            if (d == 0) p.part_lse[at] = r.l != r.l ? 0.f : r.l > 0.f ? r.m * kLog2e + log2f(r.l) + kLift : -INFINITY;
        }
    }
}

// NQ: groups of 8 query rows a tile.
template <int MODE, int D, int NQ>
__global__ void __launch_bounds__(kThreads, NQ == 1 ? kCtas : 2)
kv_attn_decode_kernel(const __grid_constant__ DecodeArgs p, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap) {
    constexpr int NS = kStages<D>;
    constexpr int kHalf = kTile * D;  // bytes of K (or V) a stage
    constexpr int KS = D / 16;        // k-steps of the first product
    constexpr int MT = D / 16;        // 16-value tiles of the second
    constexpr int RT = 8 * NQ;        // rows a tile
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t* stages = smem;                                            // [NS][2][kHalf]
    float* join = reinterpret_cast<float*>(smem + NS * 2 * kHalf);     // [RT][D]
    __shared__ __align__(8) uint64_t full[NS], empty[NS], meta_full[2], meta_empty[2];
    __shared__ ItemMeta meta[2];
    __shared__ BlockScales scales[2][kBlocksMax];
    __shared__ int64_t prefix[kThreads + 1];
    __shared__ float join_m[kConsumers][RT], join_l[kConsumers][RT];
    __shared__ int failed;  // a consumer's wait gave up: all leave together, at a barrier
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    if (tid == 0) {
        failed = 0;
        for (int i = 0; i < NS; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&meta_full[i], 1);
            mbar_init(&meta_empty[i], kConsumers);
        }
        mbar_init_fence();
    }
    pdl_launch_dependents();
    if (!p.beside) pdl_wait();

    // items before each thread's run of sequences
    const int G = p.a.Hq / p.c.H;
    const int per = (p.st.S + kThreads - 1) / kThreads;
    {
        int64_t mine = 0;
        for (int i = 0; i < per; ++i) {
            const int s = tid * per + i;
            if (s >= p.st.S) break;
            const SeqWork w = seq_work(p, s);
            mine += static_cast<int64_t>(w.tiles) * w.chunks;
        }
        prefix[tid + 1] = mine;
        if (tid == 0) prefix[0] = 0;
        __syncthreads();
        if (warp == 0) {  // five values a lane
            int64_t v[kThreads / 32], sum = 0;
#pragma unroll
            for (int i = 0; i < kThreads / 32; ++i) {
                sum += prefix[lane * (kThreads / 32) + i + 1];
                v[i] = sum;
            }
            int64_t before = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t n = __shfl_up_sync(0xffffffffu, before, o);
                if (lane >= o) before += n;
            }
            before -= sum;
#pragma unroll
            for (int i = 0; i < kThreads / 32; ++i) prefix[lane * (kThreads / 32) + i + 1] = before + v[i];
        }
        __syncthreads();
    }
    const int64_t total = prefix[kThreads] * p.c.H;
    bool ok = true;

    if (warp == kConsumers) {
        // ------------------------------------------------------------ producer
        int stage = 0;
        uint32_t phase = 0;
        const int box = p.c.block < kTile ? p.c.block : kTile;
        // everything about an item but its codes, into a slot that the consumers are done with
        auto prepare = [&](int64_t w, int it) {
            const int slot = it & 1;
            ok = mbar_wait(&meta_empty[slot], ((it >> 1) & 1) ^ 1, 0x61);
            if (!ok) return;
            // the sequence: its thread's run, then the sequence in the run
            const int64_t u = w / p.c.H;
            const int h = static_cast<int>(w - u * p.c.H);
            int lo = 0, hi = kThreads;
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (prefix[mid] <= u) lo = mid; else hi = mid;
            }
            int64_t left = u - prefix[lo];
            int s = lo * per;
            SeqWork sw = seq_work(p, s);
            while (left >= static_cast<int64_t>(sw.tiles) * sw.chunks) {
                left -= static_cast<int64_t>(sw.tiles) * sw.chunks;
                sw = seq_work(p, ++s);
            }
            const int tile = sw.tiles == 1 ? 0 : static_cast<int>(left / sw.chunks);
            const int chunk = static_cast<int>(left - static_cast<int64_t>(tile) * sw.chunks);
            const int f0 = tile * RT;
            const int64_t seq_rows = static_cast<int64_t>(sw.span.n) * G;
            const int rows = seq_rows - f0 < RT ? static_cast<int>(seq_rows - f0) : RT;
            const int p0 = sw.span.first + f0 / G, p1 = sw.span.first + (f0 + rows - 1) / G;  // places of its first and last row
            int t0 = sw.lo + chunk * sw.chunk;
            int t1 = t0 + sw.chunk < sw.span.len ? t0 + sw.chunk : sw.span.len;
            int lo_max = 0, hi_min = sw.span.len, lo_min = 0, hi_max = sw.span.len;
            if (p.a.causal) {
                hi_min = p0 + 1 < hi_min ? p0 + 1 : hi_min;
                hi_max = p1 + 1 < hi_max ? p1 + 1 : hi_max;
                if (p.a.window > 0) {
                    lo_max = p1 + 1 > p.a.window ? p1 + 1 - p.a.window : 0;
                    lo_min = p0 + 1 > p.a.window ? p0 + 1 - p.a.window : 0;
                }
            }
            if (t1 > hi_max) t1 = hi_max;
            if (t0 < lo_min / kTile * kTile) t0 = lo_min / kTile * kTile;
            if (t1 < t0) t1 = t0;
            const int block0 = t0 / p.c.block;
            const int blocks = t1 > t0 ? (t1 - 1) / p.c.block - block0 + 1 : 0;
            // the consumers will ask for the queries when they have joined the item before: touch them
            // (a row of D bf16 is D / 64 lines of 128 bytes)
            for (int i = lane; i < rows * (D / 64); i += 32) {
                const int f = f0 + i / (D / 64);
                const uint16_t* q = static_cast<const uint16_t*>(p.a.q) + (sw.span.row0 + f / G) * p.a.q_stride +
                                    (static_cast<int64_t>(h) * G + f % G) * D + i % (D / 64) * 64;
                asm volatile("{\n\t.reg .b32 unused;\n\tld.global.nc.b32 unused, [%0];\n\t}" ::"l"(q));
            }
            float vmax = 0.f;
            float vs_of[(kBlocksMax + 31) / 32];
#pragma unroll
            for (int i = 0; i < (kBlocksMax + 31) / 32; ++i) {
                const int b = lane + 32 * i;
                vs_of[i] = 0.f;
                if (b < blocks) {
                    // blocks in front of every row's window only share a stage with those in it
                    const int page = (block0 + b + 1) * p.c.block > lo_min ? page_of(p.st, p.c, s, block0 + b) : -1;
                    float ks = -1.f;
                    if (page >= 0) {
                        const int64_t ph = static_cast<int64_t>(page) * p.c.H + h;
                        ks = __ldg(p.c.k_scales + ph);
                        vs_of[i] = __ldg(p.c.v_scales + ph);
                    }
                    scales[slot][b].ks = ks;
                    scales[slot][b].page = page;
                    vmax = fmaxf(vmax, vs_of[i]);
                }
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, o));
            bool wide = false;
#pragma unroll
            for (int i = 0; i < (kBlocksMax + 31) / 32; ++i) {
                const int b = lane + 32 * i;
                if (b < blocks) {
                    const float lg = vs_of[i] > 0.f ? log2f(vs_of[i]) - log2f(vmax) : kLgZero;
                    wide |= vs_of[i] > 0.f && lg < kLgWide;
                    scales[slot][b].lg = lg;
                    scales[slot][b].inv = exp2f(-lg);
                }
            }
            wide = __any_sync(0xffffffffu, wide);
            if (lane == 0) {
                ItemMeta& m = meta[slot];
                m.row0 = sw.span.row0;
                m.direct = sw.chunks == 1;
                m.h = h;
                m.s = s;
                m.f0 = f0;
                m.rows = rows;
                m.first = sw.span.first;
                m.len = sw.span.len;
                m.t0 = t0;
                m.t1 = t1;
                m.lo_max = lo_max;
                m.hi_min = hi_min;
                m.chunk = chunk;
                m.block0 = block0;
                m.vmax = vmax;
                m.wide = wide;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&meta_full[slot]);
        };
        if (blockIdx.x < total) prepare(blockIdx.x, 0);
        int it = 0;
        for (int64_t w = blockIdx.x; ok && w < total; w += gridDim.x, ++it) {
            const int slot = it & 1, t0 = meta[slot].t0, t1 = meta[slot].wide ? t0 : meta[slot].t1;
            const int block0 = meta[slot].block0, h = meta[slot].h;
            for (int t = t0; ok && t < t1; t += kTile) {
                ok = mbar_wait(&empty[stage], phase ^ 1, 0x62);
                if (!ok) break;
                if (lane == 0) {
                    uint8_t* k = stages + stage * 2 * kHalf;
                    uint8_t* v = k + kHalf;
                    int boxes = 0;
                    for (int j = t; j < t + kTile && j < t1; j += box)
                        boxes += scales[slot][j / p.c.block - block0].page >= 0;
                    mbar_expect_tx(&full[stage], static_cast<uint32_t>(2 * boxes * box * D));
                    for (int j = t; j < t + kTile && j < t1; j += box) {
                        const int page = scales[slot][j / p.c.block - block0].page;
                        if (page < 0) continue;
                        const int ph = page * p.c.H + h;
                        tma_load_3d(k + (j - t) * D, &kmap, &full[stage], 0, j % p.c.block, ph);
                        tma_load_3d(v + (j - t) * D, &vmap, &full[stage], 0, j % p.c.block, ph);
                    }
                }
                __syncwarp();
                if (++stage == NS) { stage = 0; phase ^= 1; }
            }
            // the ring is full of this item's last stages: the next one's lookups cost no copies in flight
            if (ok && w + gridDim.x < total) prepare(w + gridDim.x, it + 1);
        }
        if (!ok)  // a wait gave up: let the copies in flight land before the CTA ends
            for (int i = 0; i < NS; ++i) mbar_wait(&full[i], phase ^ (i >= stage), 0x63, 10000000);
    } else {
        // ----------------------------------------------------------- consumers
        const int g = lane >> 2, t4 = lane & 3;
        // byte offsets of the lane's fragments in a warp's 32 tokens: 16-byte pieces of token rows, swizzled;
        // the row's low bits are g (keys) or 2 t4 and 2 t4 + 1 (values), the rest are constants
        uint32_t k_at[D / 64], v_at[2];
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
            k_at[i] = D == 128 ? g * 128 + ((2 * t4 + i) ^ g) * 16 : g * 64 + (t4 ^ (g >> 1 & 3)) * 16;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int row = 2 * t4 + q;
            v_at[q] = D == 128 ? row * 128 + (g ^ row) * 16 : row * 64 + ((g >> 1) ^ (row >> 1 & 3)) * 16 + (g & 1) * 8;
        }
        const int pair = warp >> 1;  // warps 0, 1 take an item's even stages, 2, 3 the odd ones; 32 tokens a warp
        uint32_t before = 0;         // stages of the items before
        int it = 0;
        for (int64_t w = blockIdx.x; ok && w < total; w += gridDim.x, ++it) {
            const int slot = it & 1;
            ok = mbar_wait(&meta_full[slot], (it >> 1) & 1, 0x64);
            if (!ok) failed = 1;
            asm volatile("bar.sync 1, 128;" ::: "memory");
            if (failed) break;
            const ItemMeta& m = meta[slot];
            if (m.wide) {
                static_assert(sizeof(PlainScratch<D>) <= RT * D * sizeof(float), "");
                wide_item<MODE, D>(p, m, *reinterpret_cast<PlainScratch<D>*>(join));
                asm volatile("bar.sync 1, 128;" ::: "memory");
                if (lane == 0) mbar_arrive(&meta_empty[slot]);
                continue;
            }
            // queries as B operands: lane 4 g + t4 holds values t4 * D / 4 .. of row g (of each group of 8)
            uint32_t qb[NQ][KS][2];
            float zc[NQ][2];               // of the lane's two score columns, rows 2 t4 and 2 t4 + 1
            int col_lo[NQ][2], col_hi[NQ][2];
            bool bad[NQ][2];
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                uint4 raw[D / 32];
                const int row = 8 * n + g;
#pragma unroll
                for (int i = 0; i < D / 32; ++i) raw[i] = make_uint4(0, 0, 0, 0);
                if (row < m.rows) {
                    const int f = m.f0 + row, tok = f / G;
                    const uint4* q = reinterpret_cast<const uint4*>(
                        static_cast<const uint16_t*>(p.a.q) + (m.row0 + tok) * p.a.q_stride +
                        (static_cast<int64_t>(m.h) * G + f % G) * D + t4 * (D / 4));
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) raw[i] = __ldg(q + i);
                }
                uint32_t most = 0;
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    const uint32_t u[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) most = max(most, max((u[j] << 16) & 0x7FFFFFFFu, u[j] & 0x7FFF0000u));
                }
                most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
                most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
                const uint32_t ex = row_exponent(most);
                const float down = pow2_bits(254u - ex);
                // word i, 16-bit pairs: values 8 i + {0, 1}, {2, 3} are k-step 2 i's b0 and b1 pairs, and so on
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    const uint32_t u[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        qb[n][2 * i + j / 2][j & 1] = f2_to_h2(__uint_as_float(u[j] << 16) * down,
                                                               __uint_as_float(u[j] & 0xFFFF0000u) * down);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int c = 2 * t4 + e;  // column of the group
                    const uint32_t ex_c = __shfl_sync(0xffffffffu, ex, 4 * c);
                    bad[n][e] = __shfl_sync(0xffffffffu, most, 4 * c) >= 0x7F800000u;
                    zc[n][e] = p.a.scale * kLog2e * pow2_bits(ex_c);
                    col_lo[n][e] = 0;
                    col_hi[n][e] = m.len;
                    if (p.a.causal && 8 * n + c < m.rows) {
                        const int pos = m.first + (m.f0 + 8 * n + c) / G;
                        col_hi[n][e] = pos + 1 < m.len ? pos + 1 : m.len;
                        if (p.a.window > 0 && pos + 1 > p.a.window) col_lo[n][e] = pos + 1 - p.a.window;
                    }
                }
            }
            float o[NQ][MT][4];  // (value g, rows 2 t4 and + 1), (value g + 8, the same) of each 16-value tile
            float ref[NQ][2], l[NQ][2];
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
#pragma unroll
                for (int i = 0; i < MT; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
                ref[n][0] = ref[n][1] = -INFINITY;
                l[n][0] = l[n][1] = 0.f;
            }

            const int stages_here = (m.t1 - m.t0 + kTile - 1) / kTile;
            for (int n_stage = pair; n_stage < stages_here; n_stage += 2) {
                const int stage = (before + n_stage) % NS;
                if (!mbar_wait(&full[stage], (before + n_stage) / NS & 1, 0x65)) {
                    failed = 1;
                    break;
                }
                const int j0 = m.t0 + n_stage * kTile + 32 * (warp & 1);
                const uint8_t* kt = stages + stage * 2 * kHalf + 32 * (warp & 1) * D;
                const uint8_t* vt = kt + kHalf;
                // the scales of the two halves of 16 tokens; a half behind the end or of a bad page is not seen
                BlockScales bs[2];
                bool seen[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int j = j0 + 16 * x;
                    bs[x] = scales[slot][j < m.t1 ? (j >> p.lg_block) - m.block0 : 0];
                    seen[x] = j < m.t1 && bs[x].ks >= 0.f;
                }
                // scores of 16 tokens (x) by 8 rows: (token g, rows 2 t4 and + 1), (token g + 8, the same)
                float c[2][NQ][4];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    uint4 kw[2][D / 64];
#pragma unroll
                    for (int h2 = 0; h2 < 2; ++h2) {
#pragma unroll
                        for (int i = 0; i < D / 64; ++i)
                            kw[h2][i] = *reinterpret_cast<const uint4*>(kt + k_at[i] + (16 * x + 8 * h2) * D);
                    }
#pragma unroll
                    for (int n = 0; n < NQ; ++n) c[x][n][0] = c[x][n][1] = c[x][n][2] = c[x][n][3] = 0.f;
#pragma unroll
                    for (int i = 0; i < D / 64; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t w0 = j == 0 ? kw[0][i].x : j == 1 ? kw[0][i].y : j == 2 ? kw[0][i].z : kw[0][i].w;
                            const uint32_t w1 = j == 0 ? kw[1][i].x : j == 1 ? kw[1][i].y : j == 2 ? kw[1][i].z : kw[1][i].w;
                            const uint32_t y0 = prepare_word<MODE>(w0), y1 = prepare_word<MODE>(w1);
                            const uint32_t a0 = pair_lo_h2<MODE>(y0), a1 = pair_lo_h2<MODE>(y1);
                            const uint32_t a2 = pair_hi_h2<MODE>(y0), a3 = pair_hi_h2<MODE>(y1);
                            const int ks = 4 * i + j;
#pragma unroll
                            for (int n = 0; n < NQ; ++n) mma_f16_16816(c[x][n], a0, a1, a2, a3, qb[n][ks][0], qb[n][ks][1]);
                        }
                }
                // values: tokens 2 t4, 2 t4 + 1 and 8 + 2 t4, 9 + 2 t4 of each 16; bytes (D / 8) g + i
                uint32_t v[2][4][D / 32];
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint8_t* at = vt + v_at[q & 1] + (16 * x + 8 * (q >> 1)) * D;
                        if constexpr (D == 128) {
                            const uint4 u = *reinterpret_cast<const uint4*>(at);
                            v[x][q][0] = u.x; v[x][q][1] = u.y; v[x][q][2] = u.z; v[x][q][3] = u.w;
                        } else {
                            const uint2 u = *reinterpret_cast<const uint2*>(at);
                            v[x][q][0] = u.x; v[x][q][1] = u.y;
                        }
                    }
                const bool whole = seen[0] && seen[1] && j0 >= m.lo_max && j0 + 32 <= m.hi_min;
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int n = 0; n < NQ; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) c[x][n][e] = fmaf(c[x][n][e], zc[n][e & 1] * bs[x].ks, bs[x].lg);
                if (!whole) {
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int n = 0; n < NQ; ++n)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int j = j0 + 16 * x + g + 8 * (e >> 1);
                                if (!seen[x] || j < col_lo[n][e & 1] || j >= col_hi[n][e & 1]) c[x][n][e] = -INFINITY;
                            }
                    if (MODE == NV_KV_E4M3) {  // a slot behind the last token, or of no page, may hold a NaN code
#pragma unroll
                        for (int x = 0; x < 2; ++x)
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                if (!seen[x] || j0 + 16 * x + 8 * (q >> 1) + 2 * t4 + (q & 1) >= m.len)
#pragma unroll
                                    for (int i = 0; i < D / 32; ++i) v[x][q][i] = 0;
                    }
                }
                // a reference is the same in all lanes of a column; it moves when one of them passes it by kSlack
                bool grow = false;
#pragma unroll
                for (int n = 0; n < NQ; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        grow |= fmaxf(fmaxf(c[0][n][e], c[0][n][e + 2]), fmaxf(c[1][n][e], c[1][n][e + 2])) > ref[n][e] + kSlack;
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int n = 0; n < NQ; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float mx = fmaxf(fmaxf(c[0][n][e], c[0][n][e + 2]), fmaxf(c[1][n][e], c[1][n][e + 2]));
                            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                            // each row by itself: its result must not depend on its neighbours
                            const bool up = mx > ref[n][e] + kSlack;
                            const float f = up ? exp2f(ref[n][e] - mx) : 1.f;
                            ref[n][e] = up ? mx : ref[n][e];
                            l[n][e] *= f;
#pragma unroll
                            for (int i = 0; i < MT; ++i) {
                                o[n][i][e] *= f;
                                o[n][i][e + 2] *= f;
                            }
                        }
                }
                uint32_t pb[2][NQ][2];  // weights as B operands: row g, tokens 2 t4, + 1 and 8 + 2 t4, + 1
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                    const float base0 = kLift - (ref[n][0] > -INFINITY ? ref[n][0] : 0.f);
                    const float base1 = kLift - (ref[n][1] > -INFINITY ? ref[n][1] : 0.f);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float w0 = exp2_approx(c[x][n][0] + base0), w1 = exp2_approx(c[x][n][1] + base1);
                        const float w2 = exp2_approx(c[x][n][2] + base0), w3 = exp2_approx(c[x][n][3] + base1);
                        l[n][0] = fmaf(w0 + w2, bs[x].inv, l[n][0]);
                        l[n][1] = fmaf(w1 + w3, bs[x].inv, l[n][1]);
                        pb[x][n][0] = transpose_8x8(f2_to_h2(w0, w1));
                        pb[x][n][1] = transpose_8x8(f2_to_h2(w2, w3));
                    }
                }
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) {
                        const uint32_t a0 = prepare_word<MODE>(v[x][0][i]), a1 = prepare_word<MODE>(v[x][1][i]);
                        const uint32_t b0 = prepare_word<MODE>(v[x][2][i]), b1 = prepare_word<MODE>(v[x][3][i]);
#pragma unroll
                        for (int half = 0; half < 2; ++half) {  // bytes 2 half and 2 half + 1 of the word: values g and g + 8 of a tile
                            const uint32_t y0 = tc::prmt(a0, a1, half ? 0x7362 : 0x5140), y1 = tc::prmt(b0, b1, half ? 0x7362 : 0x5140);
                            const uint32_t f0 = pair_lo_h2<MODE>(y0), f1 = pair_hi_h2<MODE>(y0);
                            const uint32_t f2 = pair_lo_h2<MODE>(y1), f3 = pair_hi_h2<MODE>(y1);
#pragma unroll
                            for (int n = 0; n < NQ; ++n)
                                mma_f16_16816(o[n][2 * i + half], f0, f1, f2, f3, pb[x][n][0], pb[x][n][1]);
                        }
                    }
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[stage]);
            }
            before += stages_here;
            // join the four warps: references and sums first, then the outputs in warp order
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float sum = l[n][e];
                    sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                    if (g == 0) {
                        join_m[warp][8 * n + 2 * t4 + e] = ref[n][e];
                        join_l[warp][8 * n + 2 * t4 + e] = bad[n][e] ? NAN : sum;
                    }
                }
            asm volatile("bar.sync 1, 128;" ::: "memory");
            // The buffer holds RT rows: as many warps' tiles at once as fit (an item of RT / 2 rows takes two
            // rounds), the later warps' first; then they add in turn.
            const int fit = RT / m.rows < kConsumers ? RT / m.rows >= 2 ? 2 : 1 : kConsumers;
            for (int first = kConsumers - fit; first >= 0; first -= fit) {
                if (warp >= first && warp < first + fit) {
#pragma unroll
                    for (int n = 0; n < NQ; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int row = 8 * n + 2 * t4 + e;
                            if (row >= m.rows) continue;
                            float top = -INFINITY;
#pragma unroll
                            for (int i = 0; i < kConsumers; ++i) top = fmaxf(top, join_m[i][row]);
                            const float f = top > -INFINITY ? exp2f(ref[n][e] - top) : 0.f;
                            float* dst = join + ((warp - first) * m.rows + row) * D + (D / 8) * g;
#pragma unroll
                            for (int i = 0; i < MT; i += 2) {  // tile i: values (D / 8) g + 2 i and + 1
                                float4 x = make_float4(o[n][i][e] * f, o[n][i][e + 2] * f, o[n][i + 1][e] * f, o[n][i + 1][e + 2] * f);
                                if (first + fit < kConsumers) {
                                    const float4 y = *reinterpret_cast<const float4*>(dst + 2 * i);
                                    x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
                                }
                                *reinterpret_cast<float4*>(dst + 2 * i) = x;
                            }
                        }
                }
                asm volatile("bar.sync 1, 128;" ::: "memory");
            }
            // each warp finishes every fourth row
            for (int row = warp; row < m.rows; row += kConsumers) {
                float top = -INFINITY, sum = 0.f;
#pragma unroll
                for (int i = 0; i < kConsumers; ++i) top = fmaxf(top, join_m[i][row]);
#pragma unroll
                for (int i = 0; i < kConsumers; ++i)
                    sum += join_l[i][row] * (join_m[i][row] > -INFINITY ? exp2f(join_m[i][row] - top) : (join_l[i][row] == 0.f ? 0.f : 1.f));
                const float inv = sum > 0.f || sum != sum ? m.vmax / sum : 0.f;
                const int f = m.f0 + row;
                for (int d = lane * 4; d < D; d += 128) {
                    float4 x = *reinterpret_cast<const float4*>(join + row * D + d);
                    for (int i = 1; i < fit; ++i) {
                        const float4 y = *reinterpret_cast<const float4*>(join + (i * m.rows + row) * D + d);
                        x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
                    }
                    x.x *= inv; x.y *= inv; x.z *= inv; x.w *= inv;
                    if (m.direct) {
                        uint16_t* out = static_cast<uint16_t*>(p.a.out) +
                                        ((m.row0 + f / G) * p.a.Hq + m.h * G + f % G) * D + d;
                        *reinterpret_cast<uint2*>(out) = make_uint2(tc::f2_to_bf2(x.x, x.y), tc::f2_to_bf2(x.z, x.w));
                    } else {
                        const int64_t at = part_row(p, SeqSpan{m.row0, 0, 0, 0}, m.s, m.h, f) * p.max_chunks + m.chunk;
                        *reinterpret_cast<float4*>(p.part_o + at * D + d) = x;
                        if (d == 0) p.part_lse[at] = sum != sum ? 0.f : sum > 0.f ? top + log2f(sum) : -INFINITY;
                    }
                }
            }
            asm volatile("bar.sync 1, 128;" ::: "memory");
            if (failed) break;
            if (lane == 0) mbar_arrive(&meta_empty[slot]);
        }
    }
    // what follows waits for this kernel, so this one for the kernel that it ran beside
    if (p.beside) pdl_wait();
}

// Join the chunks of the rows whose sequence took several: one CTA per row of
// partials, of one warp per eight chunks there can be; warp w sums chunks w, w + warps,
// ... in order (eight's loads in flight), then the warps' sums are added in order.
// The row's sequence is found while the kernel before still runs: what wrote the descriptor
// had ended when that one began (1 x 4096: 16.8 -> 14.7 us, 2 x 131072: 104 -> 98).
constexpr int kJoinWarps = 16, kJoinAhead = 8;
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) kv_attn_join_kernel(const __grid_constant__ DecodeArgs p) {
    __shared__ float sums[kJoinWarps][D];
    __shared__ float weights[kJoinWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int G = p.a.Hq / p.c.H;
    int64_t t;
    int s, hq;
    if (p.row_limit > 0) {
        const int f = static_cast<int>(blockIdx.x % p.row_limit);
        const int64_t sh = blockIdx.x / p.row_limit;
        s = static_cast<int>(sh / p.c.H);
        hq = static_cast<int>(sh % p.c.H) * G + f % G;
        t = clamped_start(p.st, s) + f / G;
    } else {
        t = blockIdx.x / p.a.Hq;
        hq = static_cast<int>(blockIdx.x - t * p.a.Hq);
        s = kv_find_seq(p.st, t, 1, 1, 0);
    }
    const SeqWork w = seq_work(p, s);
    pdl_launch_dependents();
    pdl_wait();
    if (t < w.span.row0 || t >= w.span.row0 + w.span.n || w.tiles == 0 || w.chunks <= 1) return;
    const int64_t at = static_cast<int64_t>(blockIdx.x) * p.max_chunks;
    constexpr int V = D / 32;  // values a lane
    float2 x[kJoinAhead][V / 2];
    float lse[kJoinAhead];
    auto load = [&](int k0) {
#pragma unroll
        for (int j = 0; j < kJoinAhead; ++j) {
            const int k = k0 + j * warps;
            lse[j] = k < w.chunks ? __ldcg(p.part_lse + at + k) : -INFINITY;
#pragma unroll
            for (int i = 0; i < V / 2; ++i)
                x[j][i] = k < w.chunks ? __ldcg(reinterpret_cast<const float2*>(p.part_o + (at + k) * D + lane * V) + i)
                                       : make_float2(0.f, 0.f);
        }
    };
    load(warp);
    float top = -INFINITY;
    for (int k = lane; k < w.chunks; k += 32) top = fmaxf(top, __ldcg(p.part_lse + at + k));
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (top == -INFINITY) top = 0.f;
    float acc[V] = {};
    float weight = 0.f;
    for (int k0 = warp; k0 < w.chunks; k0 += kJoinAhead * warps) {
        if (k0 > warp) load(k0);
#pragma unroll
        for (int j = 0; j < kJoinAhead; ++j) {
            const float e = exp2f(lse[j] - top);
            weight += e;
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                acc[2 * i] = fmaf(e, x[j][i].x, acc[2 * i]);
                acc[2 * i + 1] = fmaf(e, x[j][i].y, acc[2 * i + 1]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) sums[warp][lane * V + i] = acc[i];
    if (lane == 0) weights[warp] = weight;
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += blockDim.x) {
        float all = 0.f, x = 0.f;
        for (int i = 0; i < warps; ++i) {
            all += weights[i];
            x += sums[i][d];
        }
        static_cast<uint16_t*>(p.a.out)[(t * p.a.Hq + hq) * D + d] = f32_to_bf16_bits(all > 0.f ? x / all : 0.f);
    }
}

// K or V codes as [P * H][block][D] bytes, boxes of min(block, 64) tokens.
bool code_map(CUtensorMap* map, const uint8_t* codes, const KvCache& c) {
    EncodeTiled encode = tensor_map_encoder();
    if (!encode) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(c.D), static_cast<cuuint64_t>(c.block),
                                static_cast<cuuint64_t>(c.P) * c.H};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(c.D), static_cast<cuuint64_t>(c.D) * c.block};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(c.D), static_cast<cuuint32_t>(c.block < kTile ? c.block : kTile), 1};
    const cuuint32_t one[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(codes), dims, strides, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, c.D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int MODE, int D, int NQ>
cudaError_t launch(const DecodeArgs& p, int64_t part_rows, cudaStream_t stream, int num_sms) {
    CUtensorMap kmap, vmap;
    if (!code_map(&kmap, p.c.k_codes, p.c) || !code_map(&vmap, p.c.v_codes, p.c)) return cudaErrorInvalidValue;
    constexpr int smem = 1024 + kStages<D> * 2 * kTile * D + 8 * NQ * D * 4;
    cudaError_t e = cudaFuncSetAttribute(kv_attn_decode_kernel<MODE, D, NQ>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    // Not launched programmatically, but for the call's own kernel for many rows (512 new tokens of one sequence
    // and single ones of 31, 8192 long: 297 -> 278 us): its items are dealt out for one wave of CTAs, and those that
    // start beside the previous kernel's last ones do so unevenly (64 x 8192: 214 us so, 146 us not).
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    // one wave of resident CTAs, or as many as there can be items
    const int64_t items = (p.st.rows * (p.a.Hq / p.c.H) / p.tile_rows + p.st.S) * p.max_chunks * p.c.H;
    const int64_t wave = (NQ == 1 ? kCtas : 2) * num_sms;
    cfg.gridDim = dim3(static_cast<unsigned>(items < wave ? items : wave), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = pdl;
    cfg.numAttrs = p.beside ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, kv_attn_decode_kernel<MODE, D, NQ>, p, kmap, vmap);
    if (e != cudaSuccess || p.max_chunks <= 1) return e;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(part_rows), 1, 1);
    const int warps = (p.max_chunks + 7) / 8;
    cfg.blockDim = dim3(32 * (warps < kJoinWarps ? warps : kJoinWarps), 1, 1);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, kv_attn_join_kernel<D>, p);
}

}  // namespace

unsigned int kv_attn_decode_error_take() { return pipeline_error_take(); }

KvDecodePlan kv_decode_plan(const KvDecodeSizes& z, int num_sms) {
    KvDecodePlan r{};
    // 16-row tiles only where the 8-row ones would read the cache twice
    r.tile_rows = z.G <= 8 && (!z.only || z.most_rows <= 8) ? 8 : 16;
    // two items for every resident CTA, if the sequences are long enough
    const int64_t groups = z.S * z.H;
    int64_t target = (2 * kCtas * static_cast<int64_t>(num_sms) + groups - 1) / groups;
    r.target = static_cast<int>(target < 1 ? 1 : target > 1 << 20 ? 1 << 20 : target);
    const int64_t room = z.max_pages * z.block, cap = room < kMaxLen ? room : kMaxLen;  // no sequence is longer
    // chunks grow with the span, so the most there are is where the minimum or the maximum length binds
    int64_t most = (cap + kChunkMax - 1) / kChunkMax;
    const int64_t by_min = (cap + kChunkMin - 1) / kChunkMin;
    const int64_t by_target = by_min < r.target ? by_min : r.target;
    if (by_target > most) most = by_target;
    r.max_chunks = static_cast<int>(most < 1 ? 1 : most);
    r.row_limit = z.only ? 0 : 16;
    r.part_rows = z.only ? z.rows * z.Hq : z.S * z.H * 16;
    return r;
}

cudaError_t launch_kv_attn_decode(const KvAttn& a, const KvCache& c, const KvSteps& st, const KvDecodePlan& plan,
                                  void* workspace, bool beside, cudaStream_t stream, int num_sms) {
    const int lg_block = c.block == 16 ? 4 : c.block == 32 ? 5 : c.block == 64 ? 6 : 7;
    DecodeArgs p{a, c, st, plan.target, kChunkMax, plan.max_chunks, plan.tile_rows, lg_block, plan.row_limit, beside,
                 nullptr, nullptr};
    if (plan.max_chunks > 1) {
        p.part_o = static_cast<float*>(workspace);
        p.part_lse = p.part_o + plan.part_rows * plan.max_chunks * c.D;
    }
    const int64_t n = plan.part_rows;
    const bool i8 = c.mode == NV_KV_INT8, d128 = c.D == 128;
    if (plan.tile_rows == 8)
        return i8 ? (d128 ? launch<NV_KV_INT8, 128, 1>(p, n, stream, num_sms) : launch<NV_KV_INT8, 64, 1>(p, n, stream, num_sms))
                  : (d128 ? launch<NV_KV_E4M3, 128, 1>(p, n, stream, num_sms) : launch<NV_KV_E4M3, 64, 1>(p, n, stream, num_sms));
    return i8 ? (d128 ? launch<NV_KV_INT8, 128, 2>(p, n, stream, num_sms) : launch<NV_KV_INT8, 64, 2>(p, n, stream, num_sms))
              : (d128 ? launch<NV_KV_E4M3, 128, 2>(p, n, stream, num_sms) : launch<NV_KV_E4M3, 64, 2>(p, n, stream, num_sms));
}

}  // namespace nvq
