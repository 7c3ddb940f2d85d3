// Products of microscaled operands on the block-scaled tensor core
// (tcgen05.mma with scale factors in tensor memory): one expert's weight or
// many, grouped by the route's sort.
//
//   D[r, p] = sum_k W[e(p), r, k] x[p, k],   v[k] = code[k] * 2^(scale[k / 32] - 127)
//
// W is the 128-row operand (its rows are the accumulator's lanes) and the
// activations' rows p are the accumulator's columns, 16 to 256 of them: a
// decode step's few rows per expert cost few columns, and a weight element
// is loaded once for up to 256 rows.
//
// Work: an expert's rows form column tiles of at most 256 rows; a tile is one
// column tile times 128 weight rows, and its K range is cut into blocks of 128
// bytes of codes a row (128 E4M3 or 256 E2M1 elements); a stage of the ring is
// two of them while three such stages fit, else one.  One CTA per SM
// walks the tiles.  Warp 0 copies the codes (tensor maps, 128-byte swizzle) and
// the weights' scales (laid out once, see mx_pack_kernel), six warps the codes
// of rows in token order, two the activations' scales (into the weights' scale
// layout), warp 1 copies scales to tensor memory and issues the products, and
// warps 4-11 read the accumulator back while the next tile is computed into
// the other one.
//
// What bounds it (one GB300, weights of 128 experts, K = 6144, I = 768): few
// rows, reading the weights of the experts hit: gate/up of 16 tokens x 8, E2M1,
// 54 us, 6.5 TB/s.  One token's 78 MB take 16.4 us: its 96 tiles give 96 of the
// 152 CTAs work, and some 5 us are the launch, the tables and the first stages'
// way from memory.  Many rows, loads from memory and from L2 together: gate/up
// of 4096 tokens x 8, E4M3, 280 us, 1.5 GB from memory (67 % of its peak), 5.1 GB
// from L2, the tensor cores at 51 %; without the loads from memory it took 225,
// without the products 256.
// A plain product of 4096 x 6144 x 6144, E2M1: 51 us, 6.1 PFLOP/s, tensor cores
// at 62 %; 4.7 us of it are the last tiles' read-back.
//
// PAIR: two CTAs of a cluster form tiles of 256 weight rows, each with its own
// 128 and half of the activation rows (cta_group::2): a stage is 16 KB + 64 n
// bytes instead of 16 KB + 128 n.  Loads from L2 (about 16 TB/s over all SMs)
// bound tiles of many rows, so it takes them: gate/up of 32768 rows, E4M3, 280
// us (315 alone), the E2M1 product 4096 x 6144 x 6144 51 us (60 alone).
//
// SPLIT: where there are too few tiles for the SMs, the CTAs of a cluster share
// a tile's K range.  Each keeps its sums in its tensor memory; then every CTA
// sends them to the CTA that owns the columns (16 of them in turn, through
// distributed shared memory, into the ring's room) and adds those it owns in
// K order.  (Through global memory, with a ticket and the last CTA adding, the
// same split cost more than it gave.)
//
// The loops of warps 0 and 1 are uniform over the warp (waits end in a vote,
// one elected lane issues): as code of a single lane, the copies and products
// of a stage took 700 and 850 cycles to issue, in uniform registers a
// fraction of that.
#pragma once

#include <cuda.h>

#include "cluster.cuh"
#include "common.cuh"
#include "internal.h"
#include "tc_pipe.cuh"

namespace mr {

// Warps: 0 copies, 1 products, 2-3 scales, 4-11 read back, and for gate/up 12-17 gather.
constexpr int kExGatherWarps = 6;
__host__ __device__ constexpr int ex_threads(int op) { return op == 1 ? 384 + 32 * kExGatherWarps : 384; }
constexpr int kExMaxStages = 12;
constexpr int kExMaxN = 256;             // activation rows of a tile
constexpr int kExWBytes = 128 * 128;     // weight codes of one k-block (128 bytes a row)
// Dynamic shared memory (one CTA per SM; what gate/up's static arrays leave).
__host__ __device__ constexpr int ex_smem(int op) { return (op == 1 ? 209 : 211) * 1024; }
constexpr int kExListMax = 1536;        // column tiles in the shared list
constexpr int kExFewRows = 4;           // rows in token order that are copied one by one
constexpr int kExSfCol = 488;            // tensor-memory columns of the scale factors
constexpr int kExBuf1 = 232;             // first column of the second accumulator
// The two accumulators share columns 232-255 (256 + 256 + 24 columns of
// scale factors would not fit into 512): a tile that uses them is read back
// there first.
constexpr int kExStagePitch = 64 * 2 + 16;  // staged SwiGLU row (64 bf16), padded

enum { kExGemm = 0, kExGateUp = 1, kExDown = 2 };

struct ExpertArgs {
    CUtensorMap tm_w;        // weight codes, box of 128 rows x 128 bytes
    CUtensorMap tm_x;        // activation codes, box of 16 rows (gather: 1 row) x 128 bytes
    CUtensorMap tm_x64;      // the same in boxes of 64 rows
    const uint8_t* w_scale;  // packed: [E][row tile][k-block][512 * words]
    const uint8_t *x_scale, *x_scale_end;  // [rows][lds] bytes
    int64_t lds;
    const int32_t* sorted;   // [cap] assignment of a sorted position
    const int32_t* experts;  // [nblk] expert of a block
    void* out;               // bf16 (or fp32) rows, or E4M3 / E2M1 codes; kExDown: bf16 [assignments][R]
    uint16_t* out_low;       // kExDown: null, or the lower halves of the fp32 products, out then the upper ones
    uint8_t* out_scale;
    int64_t ldo;             // elements between output rows (kExGemm)
    const uint8_t* x;        // activation codes (rows in token order)
    int64_t ldx;
    unsigned long long wait_ns;
    int E, R, RT, KI, kb, kbytes;  // weight rows, row tiles, k-blocks, scale and code bytes per row
    int M, topk, mk, nblk, block;
    int per;                 // kExGemm: rows of a column tile
    int slices, slice_len;   // SPLIT: CTAs of a cluster, k-blocks of each
    int gather;              // x rows in token order
    int sf_vec;              // bytes that the scale rows can be read in: 16, 8, else any
    int list_cap;            // column tiles that the shared list holds (0: none, they are searched for)
    int out_fmt;             // 0 bf16, 1 MXFP8, 2 MXFP4, 3 fp32
    int flags;
};

// Scale factors: 32 rows of 16 bytes without swizzle, 8-row groups 128 bytes apart.
constexpr unsigned long long kExDescSf = ((unsigned long long)(128 >> 4) << 32) | (1ull << 46);
// 32 rows of 16 bytes to four tensor-memory columns, repeated in each of the
// four 32-lane quarters: lane l, column c holds the four scales of row 32 c + l.
// (PAIR: in both CTAs, each from its own shared memory.)
template <bool PAIR>
__device__ __forceinline__ void ex_copy_sf(uint32_t tmem, uint32_t addr) {
    if (PAIR)
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(ex_desc(kExDescSf, addr))
                     : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(ex_desc(kExDescSf, addr))
                     : "memory");
}
// Instruction descriptor without the scale selectors: E4M3 (format 0 of
// kind::mxf8f6f4) or E2M1 (format 1 of kind::mxf4), both operands K-major,
// E8M0 scales, 128 rows (PAIR: 256, 128 in each CTA), n columns.
template <bool FP4, bool PAIR>
__device__ __forceinline__ uint32_t ex_idesc(int n) {
    return ((FP4 ? 1u : 0u) << 7) | ((FP4 ? 1u : 0u) << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) |
           ((PAIR ? 2u : 1u) << 27);
}
// One k-step (32 E4M3 or 64 E2M1 elements); sel = index of its first scale in
// the 32-bit scale words of both operands.
#define EX_MMA(group, kind)                                                                                       \
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"                                                \
                 "tcgen05.mma.cta_group::" group ".kind::" kind " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d), \
                 "l"(a), "l"(b), "r"(id), "r"(sfa), "r"(sfb), "r"((uint32_t)acc)                                  \
                 : "memory")
template <bool FP4, bool PAIR>
__device__ __forceinline__ void ex_mma(uint32_t d, unsigned long long a, unsigned long long b, uint32_t idesc,
                                       uint32_t sel, uint32_t sfa, uint32_t sfb, bool acc) {
    const uint32_t id = idesc | (sel << 4) | (sel << 29);
    if (FP4 && PAIR) EX_MMA("2", "mxf4.block_scale.scale_vec::2X");
    else if (FP4) EX_MMA("1", "mxf4.block_scale.scale_vec::2X");
    else if (PAIR) EX_MMA("2", "mxf8f6f4.block_scale.scale_vec::1X");
    else EX_MMA("1", "mxf8f6f4.block_scale.scale_vec::1X");
}
#undef EX_MMA
// L2 policies of the weights: those that one tile alone reads are the first to
// go from L2, so that what is read again (activations, products on their way
// to the sum) stays.  Gate/up of 16 tokens x 8 over 128 experts, E2M1: 54.5 us
// (56.4 without), down of 64: 47.5 (50.5); for weights that two tiles read it
// would cost: gate/up of 4096 tokens, E4M3: 306 us instead of 282.
__device__ __forceinline__ uint64_t ex_policy(bool once) {
    uint64_t first, normal;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(first));
    asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(normal));
    return once ? first : normal;
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* map, int x, int y, int z, uint32_t bar,
                                            uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, "
        "%3, %4}], [%5], %6;" ::"r"(dst),
        "l"(reinterpret_cast<unsigned long long>(map)), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(policy)
        : "memory");
}
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const void* map, int x, int y, int z, int u, int v,
                                            uint32_t bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, "
        "%3, %4, %5, %6}], [%7], %8;" ::"r"(dst),
        "l"(reinterpret_cast<unsigned long long>(map)), "r"(x), "r"(y), "r"(z), "r"(u), "r"(v), "r"(bar), "l"(policy)
        : "memory");
}
// 16 bytes of global memory (bytes of them, 0 or 16; the rest zeros) into shared memory.
__device__ __forceinline__ void ex_cp_async16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// a / b for a < 2^23 (a quotient rounded to within one, then put right): the
// general division is several times longer, and the ones between the tables
// and the first copy are in every call's way.
__device__ __forceinline__ unsigned ex_div(unsigned a, unsigned b) {
    unsigned q = __float2uint_rz(__fdividef((float)a, (float)b));
    const int r = (int)(a - q * b);
    if (r < 0) --q;
    else if (r >= (int)b) ++q;
    return q;
}

// Up to 16 scale bytes of a row from any address at (the rest zeros), left of
// them in the row: out of lo and hi, the two aligned 16 bytes around them, or
// (whole false: those would leave the array) byte by byte.
__device__ __forceinline__ uint4 ex_scales16(const uint8_t* at, int left, uint4 lo, uint4 hi, bool whole) {
    const unsigned off = (unsigned)(reinterpret_cast<uintptr_t>(at) & 15u);
    uint32_t w[4];
    if (whole) {
        uint32_t x[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int i = 0; i < 6; ++i) x[i] = (off & 8u) ? x[i + 2] : x[i];
#pragma unroll
        for (int i = 0; i < 5; ++i) x[i] = (off & 4u) ? x[i + 1] : x[i];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(x[i], x[i + 1], (off & 3u) * 8u);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = 0u;
            for (int u = 0; u < 4; ++u)
                if (4 * i + u < left) w[i] |= (uint32_t)at[4 * i + u] << (8 * u);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = left - 4 * i;
        if (n < 4) w[i] = n <= 0 ? 0u : w[i] & ((1u << (8 * n)) - 1u);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The experts' column tiles, built by every CTA from the route's outputs.
struct ExTables {
    int* first;  // [E] first sorted position
    int* rows;   // [E] rows
    int* pre;    // [E + 1] column tiles before expert e
    int2* list;  // [list_cap] column tiles: first position, expert << 16 | rows
};
struct ExTile {
    int e, rt, r0, rows, n;  // expert, row tile, first position, real rows, accumulator columns
};
__device__ __forceinline__ int ex_ncol(int rows) { return (rows + kExMaxN - 1) / kExMaxN; }
// Rows of each column tile of an expert (equal shares, a multiple of 16): at
// most 256, and every tile has at least one row.
// (a pair's columns are split between its CTAs: a multiple of 32)
template <bool PAIR>
__device__ __forceinline__ int ex_round(int rows) { return PAIR ? (rows + 31) & ~31 : (rows + 15) & ~15; }
template <bool PAIR>
__device__ __forceinline__ int ex_share(int rows, int nct) {
    return ex_round<PAIR>(nct <= 1 ? rows : (rows + nct - 1) / nct);
}

// Column tile ct: of the list, or (a list that does not fit: more than some
// hundred thousand assignments) by a search over the experts.
template <bool PAIR, int OP>
__device__ __forceinline__ ExTile ex_tile(const ExTables& t, int E, int ct, int rt, bool listed, int M, int per_gemm) {
    ExTile o;
    o.rt = rt;
    if (OP == kExGemm) {  // one expert, tiles of per rows
        o.e = 0;
        o.r0 = ct * per_gemm;
        o.rows = min(per_gemm, M - o.r0);
    } else if (listed) {
        const int2 v = t.list[ct];
        o.r0 = __shfl_sync(kFull, v.x, 0);
        const int w = __shfl_sync(kFull, v.y, 0);
        o.e = w >> 16;
        o.rows = w & 0xFFFF;
    } else {
        int lo = 0, hi = E;  // pre[lo] <= ct < pre[hi]
        while (hi - lo > 1) {
            const int m = (lo + hi) >> 1;
            if (__shfl_sync(kFull, t.pre[m], 0) <= ct) lo = m;
            else hi = m;
        }
        o.e = lo;
        const int rows = t.rows[lo], nct = t.pre[lo + 1] - t.pre[lo], i = ct - t.pre[lo];
        const int per = ex_share<PAIR>(rows, nct);
        o.r0 = __shfl_sync(kFull, t.first[lo] + i * per, 0);
        o.rows = __shfl_sync(kFull, min(per, rows - i * per), 0);
    }
    o.n = ex_round<PAIR>(o.rows);
    return o;
}

// The tiles of this CTA (or pair), every nth of n, row tiles fastest: the CTAs
// at work share few activation rows and each weight is read once.
struct ExWalk {
    int ct, rt, dct, drt, RT, end;
    bool once;  // one tile, whatever the tables say (SPLIT: its CTAs meet twice)
    __device__ __forceinline__ ExWalk(int me, int n, int row_tiles, bool single)
        : ct(me / row_tiles), rt(me - me / row_tiles * row_tiles), dct(n / row_tiles),
          drt(n - n / row_tiles * row_tiles), RT(row_tiles), end(0), once(single) {}
    __device__ __forceinline__ bool more() const { return ct < end; }
    __device__ __forceinline__ void next() {
        ct = once ? end : ct + dct;
        rt += drt;
        if (rt >= RT) rt -= RT, ++ct;
    }
};

template <bool FP4, int OP, bool PAIR, bool SPLIT>
__global__ void __launch_bounds__(ex_threads(OP), 1) expert_kernel(const __grid_constant__ ExpertArgs a) {
    constexpr int kExThreads = ex_threads(OP);
    constexpr int W = FP4 ? 2 : 1;  // scale words (of 4 bytes) per row and k-block
    extern __shared__ __align__(16) unsigned char dsm[];
    __shared__ __align__(8) unsigned long long s_full[kExMaxStages], s_empty[kExMaxStages], s_tfull[2], s_tfree, s_drain;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort, s_total, s_nmax, s_warp[kExThreads / 32];
    __shared__ __align__(16) int s_f[2][OP == kExGemm ? 4 : kExMaxN];
    __shared__ int s_tok[kExGatherWarps][OP == kExGateUp ? kExMaxN : 1];  // (each gathering warp) tokens of the tile's rows
    __shared__ __align__(16) unsigned char s_act[OP == kExGateUp ? 4 * 16 * kExStagePitch : 16];
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(kFull, tid >> 5, 0);
    const bool gather = OP == kExGateUp && a.gather;
    const int rank = PAIR ? (int)cluster_rank() : 0, slice = SPLIT ? (int)cluster_rank() : 0;
    // this CTA's k-blocks
    const int kb0 = SPLIT ? slice * a.slice_len : 0, kb1 = SPLIT ? min(a.KI, kb0 + a.slice_len) : a.KI;
    const uint32_t full0 = smem_u32(&s_full[0]), empty0 = smem_u32(&s_empty[0]);

    // ---- set-up that reads nothing of the kernel before
    if (tid < kExMaxStages) {
        mbar_init(full0 + 8u * tid, (gather ? 4 : 3) + (PAIR && rank == 0 ? 1 : 0));  // (one from the peer)
        mbar_init(empty0 + 8u * tid, 1);
        if (tid < 2) mbar_init(smem_u32(&s_tfull[tid]), 1);
        if (tid == 2) mbar_init(smem_u32(&s_tfree), PAIR ? 16 : 8);
        if (tid == 3) mbar_init(smem_u32(&s_drain), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        if (tid == 4) s_abort = 0, s_nmax = 16;
    }
    if (tid == 64) {
        tma_prefetch_map(&a.tm_w);
        tma_prefetch_map(&a.tm_x);
        if (!gather) tma_prefetch_map(&a.tm_x64);
    }
    if (warp == 1) {
        if (PAIR) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_tmem))
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_tmem))
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    ExTables t;
    t.list = reinterpret_cast<int2*>(dsm);
    t.first = reinterpret_cast<int*>(t.list + a.list_cap);
    t.rows = t.first + a.E;
    t.pre = t.rows + a.E;
    if (OP != kExGemm)
        for (int e = tid; e < a.E; e += kExThreads) t.first[e] = -1, t.rows[e] = 0;
    // a pair takes two row tiles at a time, one in each CTA
    // (a cluster that splits its K range has one tile at most)
    const int of = PAIR ? 2 : SPLIT ? a.slices : 1;
    ExWalk walk((int)blockIdx.x / of, (int)gridDim.x / of, PAIR ? (a.RT + 1) >> 1 : a.RT, SPLIT);
    pdl_trigger();
    pdl_wait();
    if (OP != kExGemm) {
        // ---- the experts' runs of blocks.  A thread reads a block's expert, its neighbours', and every 16th of its
        // positions (the assignments of a block stand before its padding, so these tell to 16 rows where a run
        // ends): independent loads, one latency
        for (int b0 = 0; b0 < a.nblk; b0 += kExThreads) {
            const int b = b0 + tid;
            int e = -1, before = -1, after = -1, rows = a.block;
            if (b < a.nblk) {
                e = a.experts[b];
                if (b > 0) before = a.experts[b - 1];
                if (b + 1 < a.nblk) after = a.experts[b + 1];
                const int32_t* s = a.sorted + (int64_t)b * a.block;
#pragma unroll 4
                for (int j = 16; j < a.block; j += 16)
                    if (s[j] >= a.mk) rows = min(rows, j);
            }
            if (b0 == 0) __syncthreads();  // (the tables' initial values)
            if (e < 0 || e >= a.E) continue;
            if (before != e) t.first[e] = b * a.block;
            if (after != e) t.rows[e] = b * a.block + rows;
        }
        __syncthreads();
    }
    if (OP != kExGemm) {  // column tiles before each expert; the widest tile
        int run = 0;
        for (int e0 = 0; e0 < a.E; e0 += kExThreads) {
            const int e = e0 + tid;
            int rows = e < a.E ? t.rows[e] : 0;  // (the end of the expert's run so far)
            if (e < a.E) t.rows[e] = rows = t.first[e] >= 0 ? max(rows - t.first[e], 0) : 0;
            const int c = ex_ncol(rows);
            int v = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(kFull, v, o);
                if (lane >= o) v += u;
            }
            if (lane == 31) s_warp[warp] = v;
            const int wide = __reduce_max_sync(kFull, c > 0 ? ex_share<PAIR>(rows, c) : 0);
            if (lane == 0) atomicMax(&s_nmax, wide);
            __syncthreads();
            const int of_warp = lane < kExThreads / 32 ? s_warp[lane] : 0;
            const int before = run + (int)__reduce_add_sync(kFull, lane < warp ? of_warp : 0) + v - c;
            run += (int)__reduce_add_sync(kFull, of_warp);
            if (e < a.E) {
                t.pre[e] = before;
                for (int i = 0; i < c && before + i < a.list_cap; ++i) {
                    const int per = ex_share<PAIR>(rows, c);
                    t.list[before + i] = make_int2(t.first[e] + i * per, (e << 16) | min(per, rows - i * per));
                }
            }
            __syncthreads();
        }
        if (tid == 0) {
            t.pre[a.E] = run;
            s_total = run;
        }
    }
    tc_fence_before();
    if (PAIR) ex_cluster_sync();
    else __syncthreads();
    tc_fence_after();

    const int total = OP == kExGemm ? (a.M + a.per - 1) / a.per : __shfl_sync(kFull, s_total, 0);
    const int xrows = OP == kExGemm ? a.per : __shfl_sync(kFull, s_nmax, 0);
    const bool listed = total <= a.list_cap;
    const int H = (xrows + 127) >> 7;  // 128-row groups of the activations' scales
    const uint32_t tmem = __shfl_sync(kFull, s_tmem, 0);
    // stages of weight and activation codes, then their scale factors
    const uint32_t dyn = smem_u32(dsm);
    const uint32_t base = (dyn + (uint32_t)a.list_cap * 8u + (uint32_t)(3 * a.E + 1) * 4u + 1023u) & ~1023u;
    const uint32_t code_bytes = (uint32_t)(kExWBytes + xrows * (PAIR ? 64 : 128)), sf_bytes = (uint32_t)(W * 512 * (1 + H));
    // k-blocks that fit, in stages of D: a stage has its waits and its arrivals whatever it holds.  (One of a tile of
    // many gathered rows holds one k-block, so that every gathering warp has its own: gate/up of 2048 tokens in token
    // order, E4M3, 210 us, of stages of two 252.)
    const int fit = (int)ex_div(dyn + (uint32_t)ex_smem(OP) - base, code_bytes + sf_bytes);
    const int D = fit >= 6 && !(gather && xrows >= 128) ? 2 : 1, nst = min(kExMaxStages, D == 2 ? fit >> 1 : fit);
    const uint32_t stage_bytes = (uint32_t)D * code_bytes, sf_stage = (uint32_t)D * sf_bytes;
    const uint32_t sf_base = base + (uint32_t)nst * stage_bytes;
    walk.end = total;
    int st = 0;       // stage of the ring
    unsigned ph = 0;  // its phase
#define EX_TILE ex_tile<PAIR, OP>(t, a.E, walk.ct, PAIR ? walk.rt * 2 + rank : walk.rt, listed, a.M, xrows)

    if (warp == 0) {
        // ---- codes, and the weights' scales
        int issued = 0;
        bool ok = true;
        for (; ok && walk.more(); walk.next()) {
            const ExTile o = EX_TILE;
            // (a pair's second row tile may lie past the weight: its codes read as zeros, and no scale is read there)
            const uint8_t* ws = a.w_scale + ((int64_t)o.e * a.RT + min(o.rt, a.RT - 1)) * a.KI * (W * 512);
            const int nx = PAIR ? o.n >> 1 : o.n, rx = o.r0 + rank * nx;  // this CTA's activation rows
            const uint64_t policy = ex_policy(OP == kExGemm ? total == 1 : t.rows[o.e] <= kExMaxN);
            const unsigned tx = (unsigned)(kExWBytes + W * 512 + (gather ? 0 : nx * 128));
            for (int ki = kb0; ki < kb1; ki += D) {
                if (!ex_wait(empty0 + 8u * st, ph ^ 1u, a.wait_ns, &s_abort)) {
                    ok = false;
                    break;
                }
                const uint32_t full = full0 + 8u * st;
                uint32_t wsm = base + (uint32_t)st * stage_bytes, ssm = sf_base + (uint32_t)st * sf_stage;
                if (ex_elect()) {
                    const int nd = min(D, kb1 - ki);
                    mbar_expect_tx(full, tx * nd + (((a.flags & 2) && issued == 0) ? 16u : 0u));
                    for (int b = 0; b < nd; ++b, wsm += code_bytes, ssm += sf_bytes) {
                        const int x = (ki + b) * 128;
                        if (OP == kExGateUp) tma_load_5d(wsm, &a.tm_w, x, 0, 0, o.rt * 4, o.e, full, policy);
                        else tma_load_3d(wsm, &a.tm_w, x, o.rt * 128, o.e, full, policy);
                        bulk_load(ssm, ws + (int64_t)(ki + b) * (W * 512), W * 512, full);
                        if (!gather) {
                            int r = 0;
                            for (; r + 64 <= nx; r += 64)
                                tma_load_2d(wsm + kExWBytes + (uint32_t)r * 128u, &a.tm_x64, x, rx + r, full);
                            for (; r < nx; r += 16)
                                tma_load_2d(wsm + kExWBytes + (uint32_t)r * 128u, &a.tm_x, x, rx + r, full);
                        }
                    }
                }
                __syncwarp();
                ++issued;
                if (++st == nst) st = 0, ph ^= 1u;
            }
        }
        // after a wait that ran out: no copy stays in flight (bounded)
        if (!ok && lane == 0) {
            for (int i = 0; i < min(issued, nst); ++i) {
                if (--st < 0) st = nst - 1, ph ^= 1u;
                const unsigned long long t0 = global_ns();
                while (!mbar_try_wait(full0 + 8u * st, ph) && global_ns() - t0 < a.wait_ns / 16 + 1000) {
                }
            }
        }
    } else if (warp == 1 && PAIR && rank == 1) {
        // ---- a pair's products are issued by its first CTA: told when this CTA's operands are in place
        bool ok = true;
        const uint32_t peer = map_rank(full0, 0);
        for (; ok && walk.more(); walk.next()) {
            for (int ki = kb0; ki < kb1; ki += D) {
                if (!ex_wait(full0 + 8u * st, ph, a.wait_ns, &s_abort)) {
                    ok = false;
                    break;
                }
                // (the scales are stores of warps 2 and 3, gathered codes those of warps 12 and on.  With the arrival's
                // own release, gate/up of 4096 tokens, E4M3: 398 us, and the product 4096 x 6144 x 6144, E2M1: 67)
                if (ex_elect()) mbar_arrive_remote_shared(peer + 8u * st);
                __syncwarp();
                if (++st == nst) st = 0, ph ^= 1u;
            }
        }
    } else if (warp == 1) {
        // ---- products
        bool ok = true;
        const uint32_t sfa = tmem + kExSfCol, sfb = sfa + 4 * W;
        for (int it = 0; ok && walk.more(); walk.next(), ++it) {
            const ExTile o = EX_TILE;
            const uint32_t d = tmem + ((it & 1) ? kExBuf1 : 0);
            const uint32_t idesc = ex_idesc<FP4, PAIR>(o.n);
            if (it > 0) {
                ok = ex_wait(smem_u32(&s_tfree), (unsigned)(it - 1) & 1u, a.wait_ns, &s_abort);
                tc_fence_after();
            }
            for (int ki = kb0; ok && ki < kb1; ki += D) {
                if (!ex_wait(full0 + 8u * st, ph, a.wait_ns, &s_abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t wa = base + (uint32_t)st * stage_bytes, sa = sf_base + (uint32_t)st * sf_stage;
                if (ex_elect()) {
                    const int nd = min(D, kb1 - ki);
                    for (int b = 0; b < nd; ++b, wa += code_bytes, sa += sf_bytes) {
                        const unsigned long long da = ex_desc(kExDescCodes, wa);
                        const unsigned long long db = ex_desc(kExDescCodes, wa + kExWBytes);
#pragma unroll
                        for (int w = 0; w < W; ++w) {
                            ex_copy_sf<PAIR>(sfa + 4 * w, sa + 512 * w);
                            ex_copy_sf<PAIR>(sfb + 4 * w * H, sa + 512 * (W + w * H));
                            if (o.n > 128) ex_copy_sf<PAIR>(sfb + 4 * w * H + 4, sa + 512 * (W + w * H) + 512);
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int w = FP4 ? j >> 1 : 0;
                            const uint32_t sel = FP4 ? (uint32_t)(j & 1) * 2 : (uint32_t)j;
                            ex_mma<FP4, PAIR>(d, da + 2 * j, db + 2 * j, idesc, sel, sfa + 4 * w, sfb + 4 * w * H,
                                              ki > kb0 || b > 0 || j > 0);
                        }
                    }
                    ex_commit<PAIR>(empty0 + 8u * st);
                    if (ki + D >= kb1) ex_commit<PAIR>(smem_u32(&s_tfull[it & 1]));
                }
                __syncwarp();
                if (++st == nst) st = 0, ph ^= 1u;
            }
        }
    } else if (warp == 2 || warp == 3) {
        // ---- the activations' scales, as [32 rows][4 groups of 32 rows] words: one warp for rows 0-127 of the
        // tile, one for rows 128-255.  16 bytes of each row are read at a time (B k-blocks), one time ahead.
        bool ok = true;
        constexpr int B = 4 / W;
        const int half = warp == 2 ? 0 : 1;
        for (; ok && walk.more(); walk.next()) {
            const ExTile o = EX_TILE;
            const uint8_t* row[4];
            const int G = max(0, min(4, ((o.n + 31) >> 5) - 4 * half));  // groups of 32 rows that are this warp's
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int r = min((half * 4 + g) * 32 + lane, o.rows - 1);
                int64_t src = o.r0 + r;
                if (gather && g < G) {
                    int f = a.sorted[o.r0 + r];
                    if (f < 0 || f >= a.mk) f = 0;
                    src = f / a.topk;
                }
                row[g] = a.x_scale + src * a.lds;
            }
            auto load = [&](uint4 (&v)[4], int b) {  // b: first scale byte (rows that are read in 8 or 16 bytes)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    v[g] = make_uint4(0u, 0u, 0u, 0u);
                    if (g >= G) continue;
                    if (a.sf_vec == 16) {
                        if (b < a.kb) v[g] = ld_v4(row[g] + b);
                    } else {
                        uint2 lo = make_uint2(0u, 0u), hi = make_uint2(0u, 0u);
                        if (b < a.kb) lo = *reinterpret_cast<const uint2*>(row[g] + b);
                        if (b + 8 < a.kb) hi = *reinterpret_cast<const uint2*>(row[g] + b + 8);
                        v[g] = make_uint4(lo.x, lo.y, hi.x, hi.y);
                    }
                }
            };
            // rows that start anywhere: the two aligned 16 bytes around the ones from byte b (near: where they do not
            // leave the array), shifted into place only when they are due
            auto near = [&](int g, int b) { return row[g] + b - (reinterpret_cast<uintptr_t>(row[g] + b) & 15u); };
            auto whole = [&](const uint8_t* p) { return p >= a.x_scale && p + 32 <= a.x_scale_end; };
            auto load_any = [&](uint4 (&lo)[4], uint4 (&hi)[4], int b) {
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const uint8_t* p = near(g, b);
                    const bool get = whole(p) && g < G && b < a.kb;
                    lo[g] = get ? ld_v4(p) : make_uint4(0u, 0u, 0u, 0u);
                    hi[g] = get ? ld_v4(p + 16) : make_uint4(0u, 0u, 0u, 0u);
                }
            };
            auto shift = [&](uint4 (&v)[4], const uint4 (&lo)[4], const uint4 (&hi)[4], int b) {
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    v[g] = g < G && b < a.kb ? ex_scales16(row[g] + b, a.kb - b, lo[g], hi[g], whole(near(g, b)))
                                             : make_uint4(0u, 0u, 0u, 0u);
            };
            auto store = [&](const uint4 (&v)[4], int k0) {
#pragma unroll
                for (int s = 0; s < B; ++s) {
                    if (k0 + s >= kb1) return true;
                    const int b = D == 2 ? (k0 + s) & 1 : 0;  // its place in the stage
                    if (b == 0 && !ex_wait(empty0 + 8u * st, ph ^ 1u, a.wait_ns, &s_abort)) return false;
                    if (G > 0) {
                        const uint32_t sb = sf_base + (uint32_t)st * sf_stage + (uint32_t)b * sf_bytes +
                                            (W + half) * 512 + 16u * lane;
#pragma unroll
                        for (int w = 0; w < W; ++w) {
                            const int i = s * W + w;
                            auto word = [i](uint4 q) { return i == 0 ? q.x : i == 1 ? q.y : i == 2 ? q.z : q.w; };
                            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(sb + 512u * (uint32_t)(w * H)),
                                         "r"(word(v[0])), "r"(word(v[1])), "r"(word(v[2])), "r"(word(v[3]))
                                         : "memory");
                        }
                    }
                    if (b != D - 1 && k0 + s + 1 < kb1) continue;
                    if (G > 0) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mbar_arrive(full0 + 8u * st);
                    if (++st == nst) st = 0, ph ^= 1u;
                }
                return true;
            };
            uint4 v0[4], v1[4];
            if (a.sf_vec == 1) {
                uint4 v[4];
                load_any(v0, v1, kb0 * W * 4);
                for (int k0 = kb0; ok && k0 < kb1; k0 += B) {
                    shift(v, v0, v1, k0 * W * 4);
                    load_any(v0, v1, (k0 + B) * W * 4);
                    ok = store(v, k0);
                }
                continue;
            }
            load(v0, kb0 * W * 4);
            for (int k0 = kb0; ok && k0 < kb1; k0 += 2 * B) {
                load(v1, (k0 + B) * W * 4);
                ok = store(v0, k0);
                if (!ok || k0 + B >= kb1) break;
                load(v0, (k0 + 2 * B) * W * 4);
                ok = store(v1, k0 + B);
            }
        }
    } else if (OP == kExGateUp && warp >= 12) {
        // ---- codes of rows in token order: the stages in turn, one of up to six warps each, which copies the rows
        // (16 bytes a lane), waits for them and passes the stage on; the others' stages are under way meanwhile.
        // (With more of them in flight in one warp its proxy fence, which has to be its own, waits for all.)  A tile
        // of up to four rows, as decode steps have them, takes a tensor-map copy of each instead, which counts on
        // the stage's own barrier (one token's gate/up: 16.8 instead of 20.3 us).
        // At most nst warps: the one before it in a warp's turn tells that a stage's slot is at most one use behind,
        // as a wait by parity needs it.
        const int takers = min(kExGatherWarps, nst), which = warp - 12;
        int* tok = s_tok[which];
        const int quad = lane >> 3, chunk = lane & 7;  // this lane's row of four and 16-byte chunk
        bool ok = gather && which < takers;
        int turn = 0;  // whose stage is next
        int f[8];      // assignments of this CTA's rows lane, lane + 32, ...
        ExTile o{};
        auto fetch = [&] {
            if (!ok || !walk.more()) return;
            o = EX_TILE;
            const int nx = PAIR ? o.n >> 1 : o.n;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int i = lane + 32 * u, r = rank * nx + i;
                f[u] = i < nx && r < o.rows ? a.sorted[o.r0 + r] : a.mk;
            }
        };
        fetch();
        while (ok && walk.more()) {
            const int nx = PAIR ? o.n >> 1 : o.n;
            // (positions past the real ones take any token: their columns are not used)
            const bool mine = (unsigned)f[0] < (unsigned)a.mk;
            const int token = mine ? f[0] / a.topk : 0;
            const unsigned real = __ballot_sync(kFull, mine);
            const bool few = !PAIR && o.n == 16 && __popc(real) <= kExFewRows;
            if (!few) {
                __syncwarp();
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (lane + 32 * u < nx) tok[lane + 32 * u] = (unsigned)f[u] < (unsigned)a.mk ? f[u] / a.topk : 0;
                __syncwarp();
            }
            walk.next();
            fetch();  // the next tile's, while this one is copied
            for (int ki = kb0; ok && ki < kb1; ki += D) {
                if (turn == which) {
                    if (!ex_wait(empty0 + 8u * st, ph ^ 1u, a.wait_ns, &s_abort)) {
                        ok = false;
                        break;
                    }
                    const uint32_t full = full0 + 8u * st, xst = base + (uint32_t)st * stage_bytes + kExWBytes;
                    const int nd = min(D, kb1 - ki);
                    if (few) {
                        if (lane == 0) mbar_expect_tx(full, (unsigned)(__popc(real) * nd * 128));
                        __syncwarp();
                        if (mine)
                            for (int b = 0; b < nd; ++b)
                                tma_load_2d(xst + (uint32_t)b * code_bytes + (uint32_t)lane * 128u, &a.tm_x,
                                            (ki + b) * 128, token, full);
                        __syncwarp();
                    } else {
                        for (int b = 0; b < nd; ++b) {
                            const uint32_t xsm = xst + (uint32_t)b * code_bytes;
                            const int at = (ki + b) * 128 + chunk * 16, bytes = at < a.kbytes ? 16 : 0;
                            const uint8_t* x = a.x + (bytes ? at : 0);
#pragma unroll 4
                            for (int r = quad; r < nx; r += 4)
                                ex_cp_async16(xsm + (uint32_t)(r * 128 + ((chunk ^ (r & 7)) << 4)),
                                              x + (int64_t)tok[r] * a.ldx, bytes);
                        }
                        asm volatile("cp.async.wait_all;" ::: "memory");
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                        if (lane == 0) mbar_arrive(full);
                    }
                }
                if (++turn == takers) turn = 0;
                if (++st == nst) st = 0, ph ^= 1u;
            }
        }
    } else {
        // ---- accumulator -> outputs: warps 4-7 and 8-11 take alternate chunks of 16 columns
        const int wq = warp & 3, grp = (warp >> 2) - 1, et = tid - 128, gt = et & 127;
        const uint32_t lanes = (uint32_t)(wq * 32) << 16;
        unsigned turn = 0;  // staging buffer of the group
        const uint32_t tfree = PAIR ? map_rank(smem_u32(&s_tfree), 0) : smem_u32(&s_tfree);
        auto release = [&] {
            if (PAIR) mbar_arrive_remote(tfree);
            else mbar_arrive(tfree);
        };
        bool met = false;
        for (int it = 0; walk.more(); walk.next(), ++it) {
            const ExTile o = EX_TILE;
            int* f = s_f[it & 1];
            if (OP != kExGemm && et < o.n) f[et] = et < o.rows ? a.sorted[o.r0 + et] : a.mk;
            const bool ok = ex_wait(smem_u32(&s_tfull[it & 1]), (unsigned)(it >> 1) & 1u, a.wait_ns, &s_abort);
            const bool all_ok = ex_sync(1, 256, ok);
            if (!SPLIT && !all_ok) break;
            tc_fence_after();
            const uint32_t d = tmem + lanes + ((it & 1) ? kExBuf1 : 0);
            const int nch = o.n >> 4;
            if (SPLIT) {
                // every CTA's products are done, so its ring's room is free: [sender][its chunks of mine][16][128]
                ex_cluster_meet();
                const int most = (nch + a.slices - 1) / a.slices;
                for (int i = grp; i < nch; i += 2) {
                    const int owner = i % a.slices;
                    if (owner == slice) continue;
                    uint32_t v[16];
                    ex_ld16(v, d + (uint32_t)i * 16u);
                    const uint32_t to = map_rank(base, (unsigned)owner) +
                                        (uint32_t)((slice * most + i / a.slices) * 16 * 128 + wq * 32 + lane) * 4u;
#pragma unroll
                    for (int q = 0; q < 16; ++q)
                        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(to + 512u * q), "r"(v[q]) : "memory");
                }
                ex_cluster_meet();
                met = true;
                if (!all_ok) break;
            }
            // the shared columns first: the chunks after which the next tile may start
            const bool from_top = !SPLIT && !(it & 1) && o.n > kExBuf1;
            const int need = SPLIT ? 0 : from_top ? nch - kExBuf1 / 16 : (it & 1) ? min(2, nch) : 0;
            if (need <= grp && lane == 0) release();
            const int r = o.rt * 128 + wq * 32 + lane;
            for (int i = SPLIT ? slice + grp * a.slices : grp; i < nch; i += SPLIT ? 2 * a.slices : 2) {
                const int c0 = (from_top ? nch - 1 - i : i) * 16;
                uint32_t v[16];
                ex_ld16(v, d + (uint32_t)c0);
                if (SPLIT) {
                    const int most = (nch + a.slices - 1) / a.slices;
                    float sum[16];
#pragma unroll
                    for (int q = 0; q < 16; ++q) sum[q] = 0.0f;
                    for (int c = 0; c < a.slices; ++c) {
                        const uint32_t from = base + (uint32_t)((c * most + i / a.slices) * 16 * 128 + wq * 32 + lane) * 4u;
#pragma unroll
                        for (int q = 0; q < 16; ++q) {
                            float x = __uint_as_float(v[q]);
                            if (c != slice) asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(from + 512u * q) : "memory");
                            sum[q] = __fadd_rn(sum[q], x);
                        }
                    }
#pragma unroll
                    for (int q = 0; q < 16; ++q) v[q] = __float_as_uint(sum[q]);
                }
                if (i < need && i + 2 >= need) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) release();
                }
                if (OP == kExGemm) {
                    const int64_t at = (int64_t)(o.r0 + c0) * a.ldo + r;
                    const int cols = r < a.R ? o.rows - c0 : 0;
                    if (a.out_fmt == 3) {
                        float* p = static_cast<float*>(a.out) + at;
#pragma unroll
                        for (int j = 0; j < 16; ++j, p += a.ldo)
                            if (j < cols) *p = __uint_as_float(v[j]);
                    } else {
                        __nv_bfloat16* p = static_cast<__nv_bfloat16*>(a.out) + at;
#pragma unroll
                        for (int j = 0; j < 16; ++j, p += a.ldo)
                            if (j < cols) *p = __float2bfloat16_rn(__uint_as_float(v[j]));
                    }
                } else if (OP == kExDown) {
                    uint16_t* y = static_cast<uint16_t*>(a.out) + r;
                    auto rows = [&](auto put) {
#pragma unroll
                        for (int j4 = 0; j4 < 4; ++j4) {
                            const int4 as = *reinterpret_cast<const int4*>(f + c0 + 4 * j4);
                            const int s4[4] = {as.x, as.y, as.z, as.w};
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                if ((unsigned)s4[j] < (unsigned)a.mk && r < a.R)
                                    put((int64_t)s4[j] * a.R, v[4 * j4 + j]);
                        }
                    };
                    if (a.out_low != nullptr) {
                        uint16_t* low = a.out_low + r;
                        rows([&](int64_t at, uint32_t bits) { y[at] = (uint16_t)(bits >> 16), low[at] = (uint16_t)bits; });
                    } else {
                        rows([&](int64_t at, uint32_t bits) {
                            y[at] = __bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(bits)));
                        });
                    }
                } else {
                    // lanes 0-15 hold gate rows and lanes 16-31 the up rows of
                    // the same features: lanes 0-15 take the even columns,
                    // lanes 16-31 the odd ones
                    unsigned char* stage = s_act + (grp * 2 + (turn++ & 1)) * 16 * kExStagePitch;
                    const bool hi = lane >= 16;
                    unsigned char* put0 = stage + (hi ? kExStagePitch : 0) + (wq * 16 + (lane & 15)) * 2;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float mine = __uint_as_float(hi ? v[2 * j + 1] : v[2 * j]);
                        const float other = __shfl_xor_sync(kFull, __uint_as_float(hi ? v[2 * j] : v[2 * j + 1]), 16);
                        const float gv = hi ? other : mine, uv = hi ? mine : other;
                        // silu from t = e^-|g|, which cannot overflow: g / (1 + t), or g t / (1 + t) below 0.  The
                        // divisor is 1 to 2, where the quotient is good to 2 ulps.  (g / (1 + e^-g) with this quotient
                        // is 0 below -87.3, where silu times a large up value is not.  4096 tokens, E4M3: 287 us with this,
                        // 286 with that; one token 16.4 and 16.5, 17.0 with that one's quotient rounded to nearest.)
                        const float t = expf(-fabsf(gv));
                        const float s = __fdividef(gv < 0.0f ? gv * t : gv, 1.0f + t) * uv;
                        *reinterpret_cast<__nv_bfloat16*>(put0 + 2 * j * kExStagePitch) = __float2bfloat16_rn(s);
                    }
                    ex_sync(2 + grp, 128, true);
                    // 8 threads per column, 8 features each
                    const int c = gt >> 3, seg = gt & 7, i0 = o.rt * 64 + seg * 8;
                    const uint4 q = *reinterpret_cast<const uint4*>(stage + c * kExStagePitch + seg * 16);
                    const int I = a.R >> 1;
                    const bool put = (unsigned)f[c0 + c] < (unsigned)a.mk && i0 < I;
                    const int64_t p = o.r0 + c0 + c;
                    if (a.out_fmt == 0) {
                        if (put) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + p * I + i0) = q;
                    } else {
                        unsigned sb;
                        if (a.out_fmt == 1) {
                            const uint2 e8 = mx_quant_quad(q, &sb);
                            if (put) *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.out) + p * I + i0) = e8;
                        } else {
                            const uint32_t e4 = mx4_quant_quad(q, &sb);
                            if (put) *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.out) + (p * I + i0) / 2) = e4;
                        }
                        if (put && (seg & 3) == 0) a.out_scale[p * (I / 32) + i0 / 32] = (uint8_t)sb;
                    }
                }
            }
            tc_fence_before();
        }
        if (SPLIT && !met) {
            ex_cluster_meet();
            ex_cluster_meet();
        }
    }
    if (SPLIT && (warp < 4 || warp >= 12)) {  // the two meetings of the CTAs that hand sums over (tile or no tile)
        __syncwarp();
        ex_cluster_meet();
        ex_cluster_meet();
    }
    __syncthreads();
    if (PAIR) {
        if (tid == 0 && s_abort)  // a wait that ran out here ends the peer's work too
            asm volatile("st.shared::cluster.u32 [%0], 1;" ::"r"(map_rank(smem_u32(&s_abort), (unsigned)rank ^ 1u)) : "memory");
        __syncwarp();
        ex_cluster_sync();  // (no CTA leaves while its peer may still use its memory)
    }
    if (warp == 1) {
        if (s_abort) {
            // products already issued are waited for before their tensor memory goes
            if (rank == 0 && ex_elect()) ex_commit<PAIR>(smem_u32(&s_drain));
            __syncwarp();
            const unsigned long long t0 = global_ns();
            while (!mbar_try_wait(smem_u32(&s_drain), 0) && global_ns() - t0 < a.wait_ns) {
            }
        }
        __syncwarp();
        tc_fence_after();
        if (PAIR) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
        else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
#undef EX_TILE
}

}  // namespace mr
