// Product of E4M3 operands with fp32 scales per 128 (mr_fp8_gemm).
//
//   out[m, r] = sum_b xs[m, b] ws[r / 128, b] P_b[m, r],   P_b[m, r] = sum_{k in b} q[m, k] w[r, k]
//
// The scales are any fp32 numbers, so the tensor core cannot apply them: it
// computes one P_b (tcgen05.mma kind::f8f6f4, fp32) in tensor memory, and the
// read-back warps add its scaled value to sums that they keep in registers
// while it computes the next one in another buffer.  Rows of x are the
// accumulator's lanes and rows of w its columns, so a thread has one row of x
// and its scale is one number: a block costs a column one fused multiply-add.
//
// Work: persistent CTAs (or pairs of two with cta_group::2) walk the tiles of
// 128 (256) rows of x times n rows of w, row tiles fastest.  Warp 0 copies
// (tensor maps, 128-byte swizzle, a block of 128 bytes a row per stage), warp 1
// issues the products, warps 2-3 prepare the scales, warps 4-11 read back, each
// group of four half of the columns.  (At 4096 x 6144 x 6144 with 192 columns two groups
// took 134.7 us, three of a third 136.5, four 142.)  Few rows leave
// most of this idle, so tiles become narrow, stages and buffers take up to four
// blocks (one wait for all of them), products up to 64 rows are of 64, and
// where tiles are still fewer than SMs a cluster shares their K range.
//
// What bounds it: of 4096 x 6144 x 6144 (117 us captured, 2640 TFLOP/s, 1.4 of the
// bf16 rate measured here; called over and over the power cap makes it 130) a
// pair's block of K of 224 columns takes some 800 cycles: 448 for the products,
// 540 for its bytes' way from L2 (57 a cycle), 224 to read tensor memory, as many
// to add; the read-back's waits at both ends of a buffer join them.  The results'
// way out is 3 us of it.  Of few rows it is the blocks' read-back too, 305 cycles
// for one of 48 columns whatever the rows: 40 x 6144 x 6144 10.0 us (3.8 TB/s), 48
// blocks one behind another 7.1 of them; 40 x 1536 x 6144 6.7 us, 12 blocks 1.8,
// the sums' way through the cluster 2.0, start and first bytes 3.
#include "../../include/moe_route.h"
#include "fp8_plan.h"
#include "internal.h"
#include "tc_pipe.cuh"
#include "tensor_map.h"

namespace mr {

constexpr int kF8Threads = 384;

struct Fp8Args {
    CUtensorMap tm_x, tm_w;  // boxes of xrows and n (pair: n / 2) rows x 128 bytes
    const float *xs, *ws;
    void* out;
    int64_t ldxs, ldws, ldo, tiles;
    unsigned long long wait_ns;
    int M, R, KI, n, xrows, RT, nst, nbuf, out_fp32, vec, flags;
    int slices, slice_len;  // SPLIT: CTAs of a cluster, blocks of each
};

namespace {

// Instruction descriptor of kind::f8f6f4: fp32 accumulator, E4M3 operands, both K-major.
__device__ __forceinline__ uint32_t f8_idesc(int m, int n) {
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
template <bool PAIR>
__device__ __forceinline__ void f8_mma(uint32_t lead, uint32_t d, unsigned long long a, unsigned long long b,
                                       uint32_t idesc, bool acc) {
    if (PAIR)
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %5, 0;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
            "r"((uint32_t)acc), "r"(lead)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %5, 0;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
            "r"((uint32_t)acc), "r"(lead)
            : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void f8_commit(uint32_t lead, uint32_t bar) {
    if (PAIR)
        asm volatile(
            "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
            "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::
                "r"(bar),
            "h"((unsigned short)3), "r"(lead)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
            "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar), "r"(lead)
            : "memory");
}
// Two fp32 numbers in a register pair: one instruction adds both scaled, each
// rounded by itself (40 x 6144 x 6144: 10.9 -> 9.9 us, 4096: 125 -> 121).
typedef unsigned long long F8Pair;
__device__ __forceinline__ F8Pair f8_pair(uint32_t lo, uint32_t hi) {
    F8Pair r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
__device__ __forceinline__ void f8_split(F8Pair p, float& lo, float& hi) {
    uint32_t a, b;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(p));
    lo = __uint_as_float(a), hi = __uint_as_float(b);
}
__device__ __forceinline__ F8Pair f8_fma(F8Pair x, F8Pair y, F8Pair z) {
    F8Pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    return r;
}
__device__ __forceinline__ uint32_t f8_bf16(F8Pair p) {
    float lo, hi;
    f8_split(p, lo, hi);
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t f8_lds(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}
// W words of 16 contiguous bytes of every lane's row, turned among W lanes
// first, so that an instruction writes W * 16 bytes of each of 32 / W rows.
// (The requests cost, not the bytes: with 16 bytes a row the stores took 24 of
// 125 us at 4096 x 6144 x 6144.)  at: word lane % W of the first of the W
// lanes' rows; left: how many of their rows there are.
template <int W>
__device__ __forceinline__ void f8_store_words(uint8_t* at, int64_t pitch, int64_t left, uint4 (&w)[W]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < W; o *= 2) {
        const bool up = lane & o;
#pragma unroll
        for (int k = 0; k < W; ++k) {
            if (k & o) continue;
            uint32_t *lo = &w[k].x, *hi = &w[k + o].x;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t got = __shfl_xor_sync(kFull, up ? lo[q] : hi[q], o);
                if (up) lo[q] = got;
                else hi[q] = got;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < W; ++i)
        if (i < left) *reinterpret_cast<uint4*>(at + i * pitch) = w[i];
}
// The same where rows do not start on 16 bytes or columns end: words of 4 bytes
// (one number, or two of bf16), W * 4 contiguous bytes of each of 32 / W rows an
// instruction (two of bf16 on odd addresses).  cols: how many numbers there are
// from the lane's word on.  (4096 x 6143 x 6144: 130 us, each lane for itself 315;
// 1000 x 6143 x 2048: 23 and 75; with 6144 columns 112 and 17.)
template <int W>
__device__ __forceinline__ void f8_store_odd(uint8_t* at, int64_t pitch, int64_t left, uint32_t (&w)[W], int cols,
                                             bool fp32) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < W; o *= 2) {
        const bool up = lane & o;
#pragma unroll
        for (int k = 0; k < W; ++k) {
            if (k & o) continue;
            const uint32_t got = __shfl_xor_sync(kFull, up ? w[k] : w[k + o], o);
            if (up) w[k] = got;
            else w[k + o] = got;
        }
    }
    const int need = fp32 ? 1 : 2;
#pragma unroll
    for (int i = 0; i < W; ++i) {
        if (i >= left) continue;
        uint8_t* p = at + i * pitch;
        if (cols >= need && (reinterpret_cast<uintptr_t>(p) & 3u) == 0) {
            *reinterpret_cast<uint32_t*>(p) = w[i];
        } else if (!fp32) {
            if (cols >= 1) *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[i];
            if (cols >= 2) *reinterpret_cast<uint16_t*>(p + 2) = (uint16_t)(w[i] >> 16);
        }
    }
}
// N of the chunks f of 16 columns, from c0 on, to the columns from col on of the lanes' rows, the first lane's row
// row0; rows: how many of the warp's rows there are.  Whole warps call it.
template <int N, int MC>
__device__ __forceinline__ void f8_store(const Fp8Args& a, int64_t row0, int rows, int col, const F8Pair (&f)[MC][8],
                                         int c0) {
    const int lane = threadIdx.x & 31, eb = a.out_fp32 ? 4 : 2;
    const int64_t pitch = a.ldo * eb;
    if (a.vec && col + 16 * N <= a.R) {
        constexpr int W = 2 * N;  // (bf16)
        if (a.out_fp32) {
#pragma unroll
            for (int c = 0; c < N; ++c) {
                const int g = lane & ~3;
                uint4 w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float x[4];
                    f8_split(f[c0 + c][2 * i], x[0], x[1]);
                    f8_split(f[c0 + c][2 * i + 1], x[2], x[3]);
                    w[i] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                                      __float_as_uint(x[3]));
                }
                f8_store_words<4>(static_cast<uint8_t*>(a.out) + (row0 + g) * pitch + (col + 16 * c) * 4 + (lane & 3) * 16,
                                  pitch, rows - g, w);
            }
        } else {
            const int g = lane & ~(W - 1);
            uint4 w[W];
#pragma unroll
            for (int i = 0; i < W; ++i) {
                const F8Pair* p = &f[c0 + i / 2][i % 2 * 4];
                w[i] = make_uint4(f8_bf16(p[0]), f8_bf16(p[1]), f8_bf16(p[2]), f8_bf16(p[3]));
            }
            f8_store_words<W>(static_cast<uint8_t*>(a.out) + (row0 + g) * pitch + col * 2 + (lane & (W - 1)) * 16, pitch,
                              rows - g, w);
        }
        return;
    }
    if (a.out_fp32) {
#pragma unroll
        for (int c = 0; c < N; ++c) {
            const int g = lane & 16, first = col + 16 * c + (lane & 15);
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float x, y;
                f8_split(f[c0 + c][i], x, y);
                w[2 * i] = __float_as_uint(x), w[2 * i + 1] = __float_as_uint(y);
            }
            f8_store_odd<16>(static_cast<uint8_t*>(a.out) + (row0 + g) * pitch + (int64_t)first * 4, pitch, rows - g, w,
                             a.R - first, true);
        }
    } else {
        constexpr int W = 8 * N;
        const int g = lane & ~(W - 1), first = col + 2 * (lane & (W - 1));
        uint32_t w[W];
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = f8_bf16(f[c0 + i / 8][i % 8]);
        f8_store_odd<W>(static_cast<uint8_t*>(a.out) + (row0 + g) * pitch + (int64_t)first * 2, pitch, rows - g, w,
                        a.R - first, false);
    }
}

// D: blocks of a stage and of a buffer (those behind K are zeros); MC: chunks
// of 16 columns that a read-back warp takes, half of them rounded up.
// SPLIT: the CTAs of a cluster (one tile each cluster) share its K range, and
// add their sums in K order, every CTA those of the chunks that it owns.
template <bool PAIR, int D, int MC, bool SPLIT>
__global__ void __launch_bounds__(kF8Threads, 1) fp8_gemm_kernel(const __grid_constant__ Fp8Args a) {
    extern __shared__ __align__(16) unsigned char dsm[];
    __shared__ __align__(8) unsigned long long s_full[kF8MaxStages], s_empty[kF8MaxStages];
    __shared__ __align__(8) unsigned long long s_tfull[8], s_tempty[8], s_mfree[8], s_drain;
    // of the blocks in the accumulator buffers: a row's scale times that of each block of w's rows in the tile
    __shared__ float s_scale[8][3][128];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(kFull, tid >> 5, 0);
    const int rank = PAIR ? (int)cluster_rank() : 0;
    const uint32_t full0 = smem_u32(&s_full[0]), empty0 = smem_u32(&s_empty[0]);
    const uint32_t tfull0 = smem_u32(&s_tfull[0]), tempty0 = smem_u32(&s_tempty[0]);
    if (tid < kF8MaxStages) {
        mbar_init(full0 + 8u * tid, PAIR && rank == 0 ? 2 : 1);  // (one from the peer)
        mbar_init(empty0 + 8u * tid, 1);
        if (tid < 8) {
            mbar_init(tfull0 + 8u * tid, 3);  // the products, and two warps' scales
            mbar_init(tempty0 + 8u * tid, 8);
            mbar_init(smem_u32(&s_mfree[tid]), 16);  // (pair) both CTAs' buffers are free
        }
        if (tid == 8) mbar_init(smem_u32(&s_drain), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        if (tid == 9) s_abort = 0;
    }
    if (tid == 64) {
        tma_prefetch_map(&a.tm_x);
        tma_prefetch_map(&a.tm_w);
    }
    if (warp == 3) {
        // the weight's way to L2 while the kernel before ends: the first stages
        const int t0 = (int)(blockIdx.x / (SPLIT ? a.slices : PAIR ? 2 : 1)) / a.RT;
        const int k = (SPLIT ? (int)cluster_rank() * a.slice_len : 0) + lane;
        if (lane < a.nst * D && k < a.KI) ex_prefetch_2d(&a.tm_w, k * 128, t0 * a.n + rank * (a.n / 2));
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
    tc_fence_before();
    if (PAIR) ex_cluster_sync();
    else __syncthreads();
    tc_fence_after();
    pdl_trigger();
    pdl_wait();

    constexpr int of = PAIR ? 2 : 1;
    const uint32_t tmem = __shfl_sync(kFull, s_tmem, 0);
    const uint32_t base = (smem_u32(dsm) + 1023u) & ~1023u;
    // a stage: D blocks, each n (pair: n / 2) rows of w and xrows of x
    const uint32_t wbytes = (uint32_t)(a.n / of) * 128u, block_bytes = wbytes + (uint32_t)a.xrows * 128u;
    const uint32_t stage_bytes = D * block_bytes;
    int st = 0;       // stage of the ring
    unsigned ph = 0;  // its phase
    int buf = 0;      // accumulator buffer
    unsigned bph = 0;
    const int64_t first = blockIdx.x / (SPLIT ? a.slices : of), step = gridDim.x / (SPLIT ? a.slices : of);
    const int slice = SPLIT ? (int)cluster_rank() : 0;
    const int k0 = SPLIT ? slice * a.slice_len : 0, k1 = SPLIT ? min(a.KI, k0 + a.slice_len) : a.KI;
    const bool half = !PAIR && a.xrows <= 64;  // products of 64 rows: four times 16 lanes
    const uint32_t lead = ex_elect() ? 1u : 0u;  // (whole warps up to here)

    bool met = false;
    // registers of the warps that copy and issue for those that keep sums: 128 x 56 + 256 x 216 of the 384 x 168
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 0) {
            // ---- copies
            int issued = 0;
            bool ok = true;
            for (int64_t t = first; ok && t < a.tiles; t += step) {
                const int ct = (int)(t / a.RT), rt = (int)(t - (int64_t)ct * a.RT);
                const int m0 = (rt * of + rank) * 128, w0 = ct * a.n + rank * (a.n / of);
                for (int ki = k0; ki < k1; ki += D) {
                    if (!ex_wait_cta(empty0 + 8u * st, ph ^ 1u, a.wait_ns, &s_abort)) {
                        ok = false;
                        break;
                    }
                    const uint32_t full = full0 + 8u * st, at = base + (uint32_t)st * stage_bytes;
                    ex_expect(lead, full, stage_bytes + (((a.flags & 2) && issued == 0) ? 16u : 0u));
#pragma unroll
                    for (int b = 0; b < D; ++b) {
                        ex_load_2d(lead, at + b * block_bytes, &a.tm_w, (ki + b) * 128, w0, full);
                        ex_load_2d(lead, at + b * block_bytes + wbytes, &a.tm_x, (ki + b) * 128, m0, full);
                    }
                    ++issued;
                    if (++st == a.nst) st = 0, ph ^= 1u;
                }
            }
            // after a wait that ran out: no copy stays in flight (bounded)
            if (!ok && lane == 0) {
                for (int i = 0; i < min(issued, a.nst); ++i) {
                    if (--st < 0) st = a.nst - 1, ph ^= 1u;
                    const unsigned long long t0 = global_ns();
                    while (!mbar_try_wait(full0 + 8u * st, ph) && global_ns() - t0 < a.wait_ns / 16 + 1000) {
                    }
                }
            }
        } else if (warp == 1 && PAIR && rank == 1) {
            // ---- a pair's products are issued by its first CTA: told when this CTA's operands are in place
            bool ok = true;
            const uint32_t peer = map_rank(full0, 0);
            for (int64_t t = first; ok && t < a.tiles; t += step) {
                for (int ki = k0; ki < k1; ki += D) {
                    if (!ex_wait_cta(full0 + 8u * st, ph, a.wait_ns, &s_abort)) {
                        ok = false;
                        break;
                    }
                    if (ex_elect()) mbar_arrive_remote_shared(peer + 8u * st);
                    __syncwarp();
                    if (++st == a.nst) st = 0, ph ^= 1u;
                }
            }
        } else if (warp == 1) {
            // ---- products, a stage's blocks side by side into each buffer in turn
            bool ok = true;
            const uint32_t idesc = f8_idesc(half ? 64 : 128 * of, a.n), mfree0 = PAIR ? smem_u32(&s_mfree[0]) : tempty0;
            for (int64_t t = first; ok && t < a.tiles; t += step) {
                for (int ki = k0; ki < k1; ki += D) {
                    // (a pair's stage is in the peer's memory too.  The buffer last: it is the one that is waited for)
                    if (!(PAIR ? ex_wait(full0 + 8u * st, ph, a.wait_ns, &s_abort)
                               : ex_wait_cta(full0 + 8u * st, ph, a.wait_ns, &s_abort)) ||
                        !ex_wait_cta(mfree0 + 8u * buf, bph ^ 1u, a.wait_ns, &s_abort)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t at = base + (uint32_t)st * stage_bytes, d = tmem + (uint32_t)(buf * D * a.n);
#pragma unroll
                    for (int b = 0; b < D; ++b) {
                        const unsigned long long dw = ex_desc(kExDescCodes, at + b * block_bytes);
                        const unsigned long long dx = ex_desc(kExDescCodes, at + b * block_bytes + wbytes);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            f8_mma<PAIR>(lead, d + (uint32_t)(b * a.n), dx + 2 * j, dw + 2 * j, idesc, j > 0);
                    }
                    f8_commit<PAIR>(lead, empty0 + 8u * st);
                    f8_commit<PAIR>(lead, tfull0 + 8u * buf);
                    if (++st == a.nst) st = 0, ph ^= 1u;
                    if (++buf == a.nbuf) buf = 0, bph ^= 1u;
                }
            }
        } else {
            // ---- scales, a stage's at a time into the slots of the accumulator buffer: each warp those of 64 rows, a
            // lane two of them
            const int last = (a.R - 1) >> 7, row = (warp - 2) * 64 + lane;
            bool ok = true;
            for (int64_t t = first; ok && t < a.tiles; t += step) {
                const int ct = (int)(t / a.RT), rt = (int)(t - (int64_t)ct * a.RT), bt = ct * a.n >> 7;
                const int64_t m = (int64_t)(rt * of + rank) * 128 + row;
                const int64_t end = (int64_t)a.M - 1;
                const float* xs[2] = {a.xs + min(m, end) * a.ldxs, a.xs + min(m + 32, end) * a.ldxs};
                const float* ws[3];
#pragma unroll
                for (int j = 0; j < 3; ++j) ws[j] = a.ws + (int64_t)min(bt + j, last) * a.ldws;
                float x[2][D], w[3][D];
                auto fetch = [&](int ki) {
#pragma unroll
                    for (int b = 0; b < D; ++b) {
                        const bool in = D == 1 || ki + b < a.KI;  // (behind K: no scale either)
#pragma unroll
                        for (int i = 0; i < 2; ++i) x[i][b] = in ? xs[i][ki + b] : 0.0f;
#pragma unroll
                        for (int j = 0; j < 3; ++j) w[j][b] = in ? ws[j][ki + b] : 0.0f;
                    }
                };
                fetch(k0);
                for (int ki = k0; ki < k1; ki += D) {
                    if (!ex_wait_cta(tempty0 + 8u * buf, bph ^ 1u, a.wait_ns, &s_abort)) {
                        ok = false;
                        break;
                    }
#pragma unroll
                    for (int b = 0; b < D; ++b)
#pragma unroll
                        for (int j = 0; j < 3; ++j)
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                s_scale[buf * D + b][j][row + 32 * i] = __fmul_rn(x[i][b], w[j][b]);
                    // (asked for before the arrival: nothing crosses it; after it 4096 x 6144 x 6144 took 1.5 % more)
                    if (ki + D < k1) fetch(ki + D);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(tfull0 + 8u * buf);
                    if (++buf == a.nbuf) buf = 0, bph ^= 1u;
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        // ---- scaled sums: two groups of four warps, each half of the columns
        // (each takes MC chunks of 16 columns; where they are more than there are, the last ones twice, and stores
        // its own: a read in a branch takes 130 cycles more)
        const int wq = warp & 3, grp = (warp >> 2) - 1, nch = a.n >> 4;
        const int c0 = min(grp * MC, nch - MC), own = grp * MC - c0;
        const uint32_t lanes = (uint32_t)(wq * 32) << 16, mfree = PAIR ? map_rank(smem_u32(&s_mfree[0]), 0) : 0u;
        bool ok = true;
        for (int64_t t = first; ok && t < a.tiles; t += step) {
            const int ct = (int)(t / a.RT), rt = (int)(t - (int64_t)ct * a.RT);
            const int row = half ? wq * 16 + (lane & 15) : wq * 32 + lane;
            // this warp's rows, and how many of them there are
            const int64_t row0 = (int64_t)(rt * of + rank) * 128 + wq * (half ? 16 : 32);
            const int rows = (int)min((int64_t)(half ? 16 : 32), a.M - row0);
            const int col0 = ct * a.n + c0 * 16;
            // the scale block of the first columns in the tile, and the chunk from which on it is the next one
            const int j0 = (col0 >> 7) - (ct * a.n >> 7), j1 = min(j0 + 1, 2), turn = 8 - ((col0 >> 4) & 7);
            const float *p0 = &s_scale[0][j0][row], *p1 = &s_scale[0][j1][row];
            F8Pair acc[MC][8];
#pragma unroll
            for (int c = 0; c < MC; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[c][i] = 0ull;
            // batches of two chunks: one is read while the one before is added, the last of a buffer (which is given
            // back once it is in registers) while the next buffer is asked for
            constexpr int N = D * MC, NB = (N + 1) / 2;
            uint32_t v[2][2][16];
            float s0[D], s1[D];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int q = 0; q < 16; ++q) v[0][i][q] = v[1][i][q] = 0u;
#pragma unroll
            for (int b = 0; b < D; ++b) s0[b] = s1[b] = 0.0f;
            auto add = [&](int i) {
#pragma unroll
                for (int j = 2 * i; j < 2 * i + 2 && j < N; ++j) {
                    const int b = j / MC, c = j % MC;
                    const uint32_t s = __float_as_uint(c < turn ? s0[b] : s1[b]), *p = v[i & 1][j & 1];
                    const F8Pair ss = f8_pair(s, s);
#pragma unroll
                    for (int q = 0; q < 8; ++q) acc[c][q] = f8_fma(f8_pair(p[2 * q], p[2 * q + 1]), ss, acc[c][q]);
                }
            };
            for (int ki = k0; ki < k1; ki += D) {
                const bool ready = mbar_peek_cta(tfull0 + 8u * buf, bph);
                add(NB - 1);  // of the buffer before (of none: zeros)
                if (!__all_sync(kFull, ready) && !ex_wait_cta(tfull0 + 8u * buf, bph, a.wait_ns, &s_abort)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem + lanes + (uint32_t)(buf * D * a.n + c0 * 16);
                auto read = [&](int i) {
#pragma unroll
                    for (int j = 2 * i; j < 2 * i + 2 && j < N; ++j)
                        ex_ld16_async(v[i & 1][j & 1], d + (uint32_t)(j / MC * a.n) + 16u * (j % MC));
                };
                read(0);
#pragma unroll
                for (int b = 0; b < D; ++b) s0[b] = p0[(buf * D + b) * 384], s1[b] = p1[(buf * D + b) * 384];
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    ex_ld_wait();
                    ex_ld_tie(v[i & 1][0]);
                    if (2 * i + 1 < N) ex_ld_tie(v[i & 1][1]);
                    if (i + 1 < NB) {
                        read(i + 1);
                        add(i);
                        continue;
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        // (relaxed: the accumulators were read, nothing written is passed on)
                        if (PAIR) mbar_arrive_remote(mfree + 8u * buf);
                        mbar_arrive(tempty0 + 8u * buf);
                    }
                }
                if (++buf == a.nbuf) buf = 0, bph ^= 1u;
            }
            if (ok) add(NB - 1);
            if (SPLIT) {
                // every CTA's products are done, so its ring's room is free: [sender][its chunks of mine][16][128]
                ex_cluster_meet();
                const int most = (nch + a.slices - 1) / a.slices, at = wq * 32 + lane;
#pragma unroll
                for (int c = 0; c < MC; ++c) {
                    const int i = c0 + c;
                    if (c < own) continue;
                    const uint32_t to = map_rank(base, (unsigned)(i % a.slices)) +
                                        (uint32_t)((slice * most + i / a.slices) * 2048 + at) * 4u;
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        float x, y;
                        f8_split(acc[c][q], x, y);
                        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 1024u * q), "f"(x) : "memory");
                        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 1024u * q + 512u), "f"(y)
                                     : "memory");
                    }
                }
                ex_cluster_meet();
                met = true;
                // (its own sums from there too, in a loop: code that runs once costs its way to the SM)
#pragma unroll 1
                for (int i = c0 + own; i < c0 + MC && ok; ++i) {
                    if (i % a.slices != slice) continue;
                    F8Pair sum[1][8];
#pragma unroll
                    for (int q = 0; q < 8; ++q) sum[0][q] = 0ull;
#pragma unroll 1
                    for (int z = 0; z < a.slices; ++z) {
                        const uint32_t from = base + (uint32_t)((z * most + i / a.slices) * 2048 + at) * 4u;
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            asm("add.rn.f32x2 %0, %0, %1;"
                                : "+l"(sum[0][q])
                                : "l"(f8_pair(f8_lds(from + 1024u * q), f8_lds(from + 1024u * q + 512u))));
                    }
                    f8_store<1>(a, row0, rows, ct * a.n + 16 * i, sum, 0);
                }
            } else if (ok) {
                // two chunks at a time (in fp32 one): 64 bytes of a row
#pragma unroll
                for (int c = 0; c < MC; c += 2) {
                    if (c + 1 < MC && c >= own) f8_store<2>(a, row0, rows, col0 + 16 * c, acc, c);
                    else if (c >= own) f8_store<1>(a, row0, rows, col0 + 16 * c, acc, c);
                    else if (c + 1 < MC && c + 1 >= own) f8_store<1>(a, row0, rows, col0 + 16 * c + 16, acc, c + 1);
                }
            }
        }
    }
    if (SPLIT && !met) {  // the two meetings of the CTAs that hand sums over
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
}

template <bool PAIR, int D, int MC, bool SPLIT>
cudaError_t launch_one(const Fp8Args& a, int grid, cudaStream_t st) {
    static int prepared[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    const auto kernel = fp8_gemm_kernel<PAIR, D, MC, SPLIT>;
    if (!__atomic_load_n(&prepared[dev], __ATOMIC_ACQUIRE)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kF8Smem);
        if (e != cudaSuccess) return e;
        __atomic_store_n(&prepared[dev], 1, __ATOMIC_RELEASE);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kF8Threads);
    cfg.dynamicSmemBytes = kF8Smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = SPLIT ? (unsigned)a.slices : 2;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = PAIR || SPLIT ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, kernel, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool SPLIT>
cudaError_t launch_single(const Fp8Plan& p, const Fp8Args& a, cudaStream_t st) {
    switch (p.D * 10 + p.mc) {
        case 41: return launch_one<false, 4, 1, SPLIT>(a, p.grid, st);
        case 42: return launch_one<false, 4, 2, SPLIT>(a, p.grid, st);
        case 21: return launch_one<false, 2, 1, SPLIT>(a, p.grid, st);
        case 22: return launch_one<false, 2, 2, SPLIT>(a, p.grid, st);
        case 23: return launch_one<false, 2, 3, SPLIT>(a, p.grid, st);
        case 24: return launch_one<false, 2, 4, SPLIT>(a, p.grid, st);
        case 14: return launch_one<false, 1, 4, SPLIT>(a, p.grid, st);
        case 16: return launch_one<false, 1, 6, SPLIT>(a, p.grid, st);
        default: return launch_one<false, 1, 7, SPLIT>(a, p.grid, st);
    }
}
cudaError_t launch_plan(const Fp8Plan& p, const Fp8Args& a, cudaStream_t st) {
    if (p.slices > 1) return launch_single<true>(p, a, st);
    if (!p.pair) return launch_single<false>(p, a, st);
    return p.mc == 6 ? launch_one<true, 1, 6, false>(a, p.grid, st) : launch_one<true, 1, 7, false>(a, p.grid, st);
}

}  // namespace

bool fp8_encode(CUtensorMap* map, const void* ptr, int K, int64_t rows, int64_t ld, int box_rows) {
    const EncodeTiled fn = encode_tiled();
    if (fn == nullptr) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)ld};
    const cuuint32_t box[2] = {128, (cuuint32_t)box_rows}, estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int launch_fp8_gemm(const Fp8GemmCall& c, cudaStream_t st, cudaError_t* err) {
    int dev = 0, sms = 0;
    if ((*err = cudaGetDevice(&dev)) != cudaSuccess ||
        (*err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
        return MR_ERR_CUDA;
    if (fp8_few(c.M)) return launch_fp8_few(c, sms, st, err);
    const Fp8Plan p = fp8_plan(c.M, c.R, c.K, sms);
    Fp8Args a{};
    if (!fp8_encode(&a.tm_x, c.x, c.K, c.M, c.ldx, p.xrows) ||
        !fp8_encode(&a.tm_w, c.w, c.K, c.R, c.ldw, p.n / (p.pair ? 2 : 1)))
        return MR_ERR_UNSUPPORTED;
    a.xs = c.xs;
    a.ws = c.ws;
    a.out = c.out;
    a.ldxs = c.ldxs;
    a.ldws = c.ldws;
    a.ldo = c.ldo;
    a.tiles = (int64_t)p.RT * p.CT;
    a.wait_ns = wait_limit_ns();
    a.M = c.M;
    a.R = c.R;
    a.KI = (c.K + 127) / 128;
    a.n = p.n;
    a.xrows = p.xrows;
    a.RT = p.RT;
    a.nst = p.nst;
    a.nbuf = p.nbuf;
    a.out_fp32 = c.out_fp32;
    a.vec = reinterpret_cast<uintptr_t>(c.out) % 16 == 0 && c.ldo % (c.out_fp32 ? 4 : 8) == 0;
    a.flags = launch_flags();
    a.slices = p.slices;
    a.slice_len = p.slice_len;
    const cudaError_t e = launch_plan(p, a, st);
    *err = e;
    return e == cudaSuccess ? MR_OK : MR_ERR_CUDA;
}

int fp8_device_error(int clear) {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_ex_timeout, sizeof(int)) != cudaSuccess) return -1;
    if (clear && v) {
        const int z = 0;
        if (cudaMemcpyToSymbol(g_ex_timeout, &z, sizeof(int)) != cudaSuccess) return -1;
    }
    return v;
}

}  // namespace mr
