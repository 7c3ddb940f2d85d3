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
// column tile times 128 weight rows, and its K range is cut into stages of
// 128 bytes of codes a row (128 E4M3 or 256 E2M1 elements).  One CTA per SM
// walks the tiles.  Warp 0 copies the codes (tensor maps, 128-byte swizzle;
// rows in token order by four-row gathers) and the weights' scales (laid out
// once, see mx_pack_kernel), warp 2 puts the activations' scales into the
// same layout, one thread of warp 1 copies scales to tensor memory and
// issues the products, and warps 4-7 read the accumulator back while the next
// tile is computed into the other one.
#pragma once

#include <cuda.h>

#include "cluster.cuh"
#include "common.cuh"
#include "internal.h"

namespace mr {

constexpr int kExThreads = 256;
constexpr int kExMaxStages = 12;
constexpr int kExMaxN = 256;             // activation rows of a tile
constexpr int kExWBytes = 128 * 128;     // one stage of weight codes
constexpr int kExSmemDyn = 219 * 1024;   // dynamic shared memory (one CTA per SM)
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
    const uint8_t* w_scale;  // packed: [E][row tile][stage][512 * words]
    const uint8_t* x_scale;  // [rows][lds] bytes
    int64_t lds;
    const int32_t* sorted;   // [cap] assignment of a sorted position
    const int32_t* experts;  // [nblk] expert of a block
    void* out;               // bf16 (or fp32) rows, or E4M3 / E2M1 codes
    uint8_t* out_scale;
    float* y;                // kExDown: [assignments][R] fp32
    int64_t ldo;             // elements between output rows (kExGemm)
    unsigned long long wait_ns;
    int E, R, RT, KI, kb;    // weight rows, row tiles, stages, scale bytes per row
    int M, topk, mk, nblk, block;
    int gather;              // x rows in token order
    int sf_words;            // the scale rows can be read as 32-bit words
    int out_fmt;             // 0 bf16, 1 MXFP8, 2 MXFP4, 3 fp32
    int flags;
};

// Set when a bounded wait of the expert kernels ran out (read by the host).
__device__ int g_ex_timeout;

__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, unsigned parity) {
    unsigned ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// Waits for the phase of this parity, at most limit_ns; a wait that runs out
// sets the device's flag and *abort, which ends every other wait of the CTA.
__device__ __forceinline__ bool ex_wait(uint32_t bar, unsigned parity, unsigned long long limit_ns,
                                        volatile int* abort) {
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = global_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (*abort) return false;
        if (global_ns() - t0 >= limit_ns) {
            *abort = 1;
            atomicExch(&g_ex_timeout, 1);
            return false;
        }
    }
    return true;
}

// Shared-memory matrix descriptor: K-major rows of 128 bytes in the 128-byte
// swizzle (8-row groups 1024 bytes apart); a k-step starts 32 bytes further.
__device__ __forceinline__ unsigned long long ex_desc_sw128(uint32_t addr) {
    return (unsigned long long)((addr >> 4) & 0x3FFFu) | (1ull << 16) | ((unsigned long long)(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}
// Scale factors: 32 rows of 16 bytes without swizzle, 8-row groups 128 bytes apart.
__device__ __forceinline__ unsigned long long ex_desc_sf(uint32_t addr) {
    return (unsigned long long)((addr >> 4) & 0x3FFFu) | ((unsigned long long)(128 >> 4) << 32) | (1ull << 46);
}
// 32 rows of 16 bytes to four tensor-memory columns, repeated in each of the
// four 32-lane quarters: lane l, column c holds the four scales of row 32 c + l.
__device__ __forceinline__ void ex_copy_sf(uint32_t tmem, uint32_t addr) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(ex_desc_sf(addr)) : "memory");
}
// Instruction descriptor without the scale selectors: E4M3 (format 0 of
// kind::mxf8f6f4) or E2M1 (format 1 of kind::mxf4), both operands K-major,
// E8M0 scales, 128 rows, n columns.
template <bool FP4>
__device__ __forceinline__ uint32_t ex_idesc(int n) {
    return ((FP4 ? 1u : 0u) << 7) | ((FP4 ? 1u : 0u) << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) | (1u << 27);
}
// One k-step (32 E4M3 or 64 E2M1 elements); sel = index of its first scale in
// the 32-bit scale words of both operands.
template <bool FP4>
__device__ __forceinline__ void ex_mma(uint32_t d, unsigned long long a, unsigned long long b, uint32_t idesc,
                                       uint32_t sel, uint32_t sfa, uint32_t sfb, bool acc) {
    const uint32_t id = idesc | (sel << 4) | (sel << 29);
    if (FP4)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
                d),
            "l"(a), "l"(b), "r"(id), "r"(sfa), "r"(sfb), "r"((uint32_t)acc)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], "
            "p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(id), "r"(sfa), "r"(sfb), "r"((uint32_t)acc)
            : "memory");
}
__device__ __forceinline__ void ex_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// 16 accumulator columns of this warp's 32 lanes.
__device__ __forceinline__ void ex_ld16(uint32_t (&v)[16], uint32_t addr) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(dst),
        "l"(reinterpret_cast<unsigned long long>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const void* map, int x, int y, int z, int u, int v,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, "
        "%6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<unsigned long long>(map)), "r"(x), "r"(y), "r"(z), "r"(u), "r"(v), "r"(bar)
        : "memory");
}
// Four rows of a tensor map (box of one row), 128 bytes each.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const void* map, int x, int r0, int r1, int r2, int r3,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<unsigned long long>(map)), "r"(x), "r"(r0), "r"(r1), "r"(r2), "r"(r3), "r"(bar)
        : "memory");
}
// Barrier of the four epilogue warps; true when ok holds in all of them.
__device__ __forceinline__ bool ex_epi_sync(bool ok) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
        "barrier.cta.red.and.pred p, 1, 128, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)ok)
        : "memory");
    return r != 0;
}

// The experts' column tiles, built by every CTA from the route's outputs.
struct ExTables {
    int* first;  // [E] first sorted position
    int* rows;   // [E] rows
    int* pre;    // [E + 1] column tiles before expert e
};
struct ExTile {
    int e, rt, r0, rows, n;  // expert, row tile, first position, real rows, accumulator columns
};
__device__ __forceinline__ int ex_ncol(int rows) { return (rows + kExMaxN - 1) / kExMaxN; }

__device__ __forceinline__ ExTile ex_tile(const ExTables& t, int E, int RT, int tile) {
    ExTile o;
    const int ct = tile / RT;
    o.rt = tile - ct * RT;
    int lo = 0, hi = E;  // pre[lo] <= ct < pre[hi]
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (t.pre[m] <= ct) lo = m;
        else hi = m;
    }
    o.e = lo;
    const int rows = t.rows[lo], nct = t.pre[lo + 1] - t.pre[lo], i = ct - t.pre[lo];
    // equal shares: per <= 256, and every tile has at least one row
    const int per = ((rows + nct - 1) / nct + 15) & ~15;
    o.r0 = t.first[lo] + i * per;
    o.rows = min(per, rows - i * per);
    o.n = (o.rows + 15) & ~15;
    return o;
}

template <bool FP4, int OP>
__global__ void __launch_bounds__(kExThreads, 1) expert_kernel(const __grid_constant__ ExpertArgs a) {
    constexpr int W = FP4 ? 2 : 1;  // scale words (of 4 bytes) per row and stage
    extern __shared__ __align__(16) unsigned char dsm[];
    __shared__ __align__(8) unsigned long long s_full[kExMaxStages], s_empty[kExMaxStages], s_tfull[2], s_tfree, s_drain;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort, s_total, s_nmax, s_warp[8];
    __shared__ int s_f[2][kExMaxN];
    __shared__ __align__(16) unsigned char s_act[OP == kExGateUp ? 2 * 16 * kExStagePitch : 16];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    // ---- set-up that reads nothing of the kernel before
    if (tid == 0) {
        for (int s = 0; s < kExMaxStages; ++s) {
            mbar_init(smem_u32(&s_full[s]), 2);
            mbar_init(smem_u32(&s_empty[s]), 1);
        }
        mbar_init(smem_u32(&s_tfull[0]), 1);
        mbar_init(smem_u32(&s_tfull[1]), 1);
        mbar_init(smem_u32(&s_tfree), 4);
        mbar_init(smem_u32(&s_drain), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        tma_prefetch_map(&a.tm_w);
        tma_prefetch_map(&a.tm_x);
        s_abort = 0;
        s_nmax = 16;
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s_tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    ExTables t;
    t.first = reinterpret_cast<int*>(dsm);
    t.rows = t.first + a.E;
    t.pre = t.rows + a.E;
    for (int e = tid; e < a.E; e += kExThreads) {
        t.first[e] = OP == kExGemm ? 0 : -1;
        t.rows[e] = OP == kExGemm ? a.M : 0;
    }
    pdl_trigger();
    pdl_wait();
    __syncthreads();

    // ---- the experts' runs of blocks: first and last block of each
    if (OP != kExGemm) {
        for (int b = tid; b < a.nblk; b += kExThreads) {
            const int e = a.experts[b];
            if (e < 0 || e >= a.E) continue;
            if (b == 0 || a.experts[b - 1] != e) t.first[e] = b * a.block;
            if (b == a.nblk - 1 || a.experts[b + 1] != e) t.rows[e] = b + 1;
        }
        __syncthreads();
        for (int e = warp; e < a.E; e += kExThreads / 32) {
            const int f = t.first[e];
            if (f < 0) continue;
            // rows of the run without the padding of its last block (the
            // assignments of a block stand before its padding)
            const int last = (t.rows[e] - 1) * a.block;
            int real = 0;
            for (int i = lane; i < a.block; i += 32) real += a.sorted[last + i] < a.mk ? 1 : 0;
            real = __reduce_add_sync(kFull, real);
            if (lane == 0) t.rows[e] = max(last - f + real, 0);
        }
        __syncthreads();
    }
    {  // column tiles before each expert; the widest tile
        int run = 0;
        for (int e0 = 0; e0 < a.E; e0 += kExThreads) {
            const int e = e0 + tid;
            const int rows = e < a.E ? t.rows[e] : 0, c = ex_ncol(rows);
            int v = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(kFull, v, o);
                if (lane >= o) v += u;
            }
            if (lane == 31) s_warp[warp] = v;
            if (c > 0) atomicMax(&s_nmax, ((rows + c - 1) / c + 15) & ~15);
            __syncthreads();
            int before = run;
            for (int w = 0; w < warp; ++w) before += s_warp[w];
            if (e < a.E) t.pre[e] = before + v - c;
            for (int w = 0; w < kExThreads / 32; ++w) run += s_warp[w];
            __syncthreads();
        }
        if (tid == 0) {
            t.pre[a.E] = run;
            s_total = run * a.RT;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();

    const int total = s_total, xrows = s_nmax;
    const int H = (xrows + 127) >> 7;  // 128-row groups of the activations' scales
    const uint32_t tmem = s_tmem;
    // stages of weight and activation codes, then their scale factors
    const uint32_t tab = (uint32_t)(3 * a.E + 1) * 4u;
    const uint32_t base = (smem_u32(dsm) + tab + 1023u) & ~1023u;
    const uint32_t code_bytes = (uint32_t)(kExWBytes + xrows * 128), sf_bytes = (uint32_t)(W * 512 * (1 + H));
    const uint32_t room = smem_u32(dsm) + (uint32_t)kExSmemDyn - base;
    const int nst = min(kExMaxStages, (int)(room / (code_bytes + sf_bytes)));
    const uint32_t sf_base = base + (uint32_t)nst * code_bytes;
    const int step = (int)gridDim.x;
    int st = 0;        // stage of the ring
    unsigned ph = 0;   // its phase

    if (warp == 0) {
        // ---- codes, and the weights' scales
        int issued = 0;
        bool ok = true;
        for (int tile = blockIdx.x; ok && tile < total; tile += step) {
            const ExTile o = ex_tile(t, a.E, a.RT, tile);
            int tok[8];
            if (OP == kExGateUp && a.gather) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int r = (lane + (i >> 2) * 32) * 4 + (i & 3);
                    int f = r < o.rows ? a.sorted[o.r0 + r] : 0;
                    if (f < 0 || f >= a.mk) f = 0;  // a padding position: any row, its column is not used
                    tok[i] = f / a.topk;
                }
            }
            const uint8_t* ws = a.w_scale + ((int64_t)o.e * a.RT + o.rt) * a.KI * (W * 512);
            for (int ki = 0; ki < a.KI; ++ki) {
                if (!__all_sync(kFull, ex_wait(smem_u32(&s_empty[st]), ph ^ 1u, a.wait_ns, &s_abort))) {
                    ok = false;
                    break;
                }
                const uint32_t full = smem_u32(&s_full[st]);
                const uint32_t ws_s = base + (uint32_t)st * code_bytes, xs_s = ws_s + kExWBytes;
                if (lane == 0) {
                    const unsigned stall = ((a.flags & 2) && issued == 0) ? 16u : 0u;
                    mbar_expect_tx(full, (unsigned)(kExWBytes + o.n * 128 + W * 512) + stall);
                    if (OP == kExGateUp) tma_load_5d(ws_s, &a.tm_w, ki * 128, 0, 0, o.rt * 4, o.e, full);
                    else tma_load_3d(ws_s, &a.tm_w, ki * 128, o.rt * 128, o.e, full);
                    bulk_load(sf_base + (uint32_t)st * sf_bytes, ws + (int64_t)ki * (W * 512), W * 512, full);
                }
                __syncwarp();
                if (OP == kExGateUp && a.gather) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int g = lane + i * 32;
                        if (g * 4 < o.n)
                            tma_gather4(xs_s + (uint32_t)g * 512u, &a.tm_x, ki * 128, tok[4 * i], tok[4 * i + 1],
                                        tok[4 * i + 2], tok[4 * i + 3], full);
                    }
                } else if (lane * 16 < o.n) {
                    tma_load_2d(xs_s + (uint32_t)lane * 2048u, &a.tm_x, ki * 128, o.r0 + lane * 16, full);
                }
                ++issued;
                if (++st == nst) st = 0, ph ^= 1u;
            }
        }
        // after a wait that ran out: no copy stays in flight (bounded)
        if (!ok && lane == 0) {
            for (int i = 0; i < min(issued, nst); ++i) {
                if (--st < 0) st = nst - 1, ph ^= 1u;
                const unsigned long long t0 = global_ns();
                while (!mbar_try_wait(smem_u32(&s_full[st]), ph) && global_ns() - t0 < a.wait_ns / 16 + 1000) {
                }
            }
        }
    } else if (warp == 1) {
        // ---- products: one thread
        if (lane == 0) {
            bool ok = true;
            int it = 0;
            for (int tile = blockIdx.x; ok && tile < total; tile += step, ++it) {
                const ExTile o = ex_tile(t, a.E, a.RT, tile);
                const uint32_t d = tmem + ((it & 1) ? kExBuf1 : 0);
                const uint32_t sfa = tmem + kExSfCol, sfb = sfa + 4 * W;
                const uint32_t idesc = ex_idesc<FP4>(o.n);
                if (it > 0) {
                    ok = ex_wait(smem_u32(&s_tfree), (unsigned)(it - 1) & 1u, a.wait_ns, &s_abort);
                    tc_fence_after();
                }
                for (int ki = 0; ok && ki < a.KI; ++ki) {
                    if (!ex_wait(smem_u32(&s_full[st]), ph, a.wait_ns, &s_abort)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t wa = base + (uint32_t)st * code_bytes, xa = wa + kExWBytes;
                    const uint32_t sa = sf_base + (uint32_t)st * sf_bytes, sb = sa + W * 512;
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        ex_copy_sf(sfa + 4 * w, sa + 512 * w);
                        for (int h = 0; h * 128 < o.n; ++h) ex_copy_sf(sfb + 4 * (w * H + h), sb + 512 * (w * H + h));
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int w = FP4 ? j >> 1 : 0;
                        const uint32_t sel = FP4 ? (uint32_t)(j & 1) * 2 : (uint32_t)j;
                        ex_mma<FP4>(d, ex_desc_sw128(wa + 32 * j), ex_desc_sw128(xa + 32 * j), idesc, sel, sfa + 4 * w,
                                    sfb + 4 * w * H, ki > 0 || j > 0);
                    }
                    ex_commit(smem_u32(&s_empty[st]));
                    if (++st == nst) st = 0, ph ^= 1u;
                }
                if (ok) ex_commit(smem_u32(&s_tfull[it & 1]));
            }
        }
        __syncwarp();
    } else if (warp == 2) {
        // ---- the activations' scales, as [32 rows][4 groups of 32 rows] words
        bool ok = true;
        constexpr int B = FP4 ? 2 : 4;  // stages read at a time: 16 bytes of each row
        for (int tile = blockIdx.x; ok && tile < total; tile += step) {
            const ExTile o = ex_tile(t, a.E, a.RT, tile);
            const uint8_t* row[8];
#pragma unroll
            for (int g = 0; g < 8; ++g) {
                const int r = min(g * 32 + lane, o.rows - 1);
                int64_t src = o.r0 + r;
                if (OP == kExGateUp && a.gather) {
                    int f = a.sorted[o.r0 + r];
                    if (f < 0 || f >= a.mk) f = 0;
                    src = f / a.topk;
                }
                row[g] = a.x_scale + src * a.lds;
            }
            const int G = (o.n + 31) >> 5;
            for (int k0 = 0; ok && k0 < a.KI; k0 += B) {
                uint32_t v[B * W][8];
#pragma unroll
                for (int i = 0; i < B * W; ++i) {
                    const int b = (k0 * W + i) * 4;  // first scale byte
#pragma unroll
                    for (int g = 0; g < 8; ++g) {
                        v[i][g] = 0u;
                        if (g >= G) continue;
                        if (a.sf_words) {
                            if (b < a.kb) v[i][g] = __ldg(reinterpret_cast<const uint32_t*>(row[g] + b));
                        } else {
                            for (int u = 0; u < 4; ++u)
                                if (b + u < a.kb) v[i][g] |= (uint32_t)__ldg(row[g] + b + u) << (8 * u);
                        }
                    }
                }
#pragma unroll
                for (int s = 0; s < B; ++s) {
                    if (k0 + s >= a.KI) break;
                    if (!__all_sync(kFull, ex_wait(smem_u32(&s_empty[st]), ph ^ 1u, a.wait_ns, &s_abort))) {
                        ok = false;
                        break;
                    }
                    const uint32_t sb = sf_base + (uint32_t)st * sf_bytes + W * 512;
#pragma unroll
                    for (int w = 0; w < W; ++w)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            if (h < H)
                                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                                 sb + 512u * (uint32_t)(w * H + h) + 16u * lane),
                                             "r"(v[s * W + w][4 * h]), "r"(v[s * W + w][4 * h + 1]),
                                             "r"(v[s * W + w][4 * h + 2]), "r"(v[s * W + w][4 * h + 3])
                                             : "memory");
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&s_full[st]));
                    if (++st == nst) st = 0, ph ^= 1u;
                }
            }
        }
    } else if (warp >= 4) {
        // ---- accumulator -> outputs
        const int wq = warp & 3, et = tid - 128;
        const uint32_t lanes = (uint32_t)(wq * 32) << 16;
        int it = 0;
        for (int tile = blockIdx.x; tile < total; tile += step, ++it) {
            const ExTile o = ex_tile(t, a.E, a.RT, tile);
            int* f = s_f[it & 1];
            if (OP != kExGemm)
                for (int c = et; c < o.n; c += 128) f[c] = c < o.rows ? a.sorted[o.r0 + c] : a.mk;
            const bool ok = ex_wait(smem_u32(&s_tfull[it & 1]), (unsigned)(it >> 1) & 1u, a.wait_ns, &s_abort);
            if (!ex_epi_sync(ok)) break;
            tc_fence_after();
            const uint32_t d = tmem + lanes + ((it & 1) ? kExBuf1 : 0);
            const int nch = o.n >> 4;
            // the shared columns first: the chunks after which the next tile may start
            const bool down_first = !(it & 1) && o.n > kExBuf1;
            const int need = down_first ? nch - kExBuf1 / 16 : (it & 1) ? min(2, nch) : 0;
            if (need == 0 && lane == 0) mbar_arrive(smem_u32(&s_tfree));
            for (int i = 0; i < nch; ++i) {
                const int ch = down_first ? nch - 1 - i : i, c0 = ch * 16;
                uint32_t v[16];
                ex_ld16(v, d + (uint32_t)c0);
                if (i + 1 == need) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&s_tfree));
                }
                if (OP == kExGemm) {
                    const int r = o.rt * 128 + wq * 32 + lane;
                    if (r < a.R) {
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (c0 + j < o.rows) {
                                const int64_t at = (int64_t)(o.r0 + c0 + j) * a.ldo + r;
                                if (a.out_fmt == 3) static_cast<float*>(a.out)[at] = __uint_as_float(v[j]);
                                else static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(__uint_as_float(v[j]));
                            }
                    }
                } else if (OP == kExDown) {
                    const int r = o.rt * 128 + wq * 32 + lane;
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const int as = f[c0 + j];
                        if (r < a.R && as >= 0 && as < a.mk) a.y[(int64_t)as * a.R + r] = __uint_as_float(v[j]);
                    }
                } else {
                    // lanes 0-15 hold gate rows and lanes 16-31 the up rows of
                    // the same features: lanes 0-15 take the even columns,
                    // lanes 16-31 the odd ones
                    unsigned char* stage = s_act + (i & 1) * 16 * kExStagePitch;
                    const bool hi = lane >= 16;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float mine = __uint_as_float(hi ? v[2 * j + 1] : v[2 * j]);
                        const float other = __shfl_xor_sync(kFull, __uint_as_float(hi ? v[2 * j] : v[2 * j + 1]), 16);
                        const float gv = hi ? other : mine, uv = hi ? mine : other;
                        const float s = gv / (1.0f + expf(-gv)) * uv;
                        *reinterpret_cast<__nv_bfloat16*>(stage + (2 * j + (hi ? 1 : 0)) * kExStagePitch +
                                                          (wq * 16 + (lane & 15)) * 2) = __float2bfloat16_rn(s);
                    }
                    ex_epi_sync(true);
                    // 8 threads per column, 8 features each
                    const int c = et >> 3, seg = et & 7, i0 = o.rt * 64 + seg * 8;
                    const uint4 q = *reinterpret_cast<const uint4*>(stage + c * kExStagePitch + seg * 16);
                    const int as = f[c0 + c], I = a.R >> 1;
                    const bool put = as >= 0 && as < a.mk && i0 < I;
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
    }
    __syncthreads();
    if (warp == 1) {
        if (s_abort && lane == 0) {
            // products already issued are waited for before their tensor memory goes
            ex_commit(smem_u32(&s_drain));
            const unsigned long long t0 = global_ns();
            while (!mbar_try_wait(smem_u32(&s_drain), 0) && global_ns() - t0 < a.wait_ns) {
            }
        }
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

}  // namespace mr
