// The expert products' launches: mr_mx_pack_scales, mr_mx_gemm,
// mr_moe_gate_up and mr_moe_down (see expert_gemm.cuh for the kernel).
#include "../../include/moe_route.h"
#include "expert_gemm.cuh"
#include "expert_plan.h"
#include "tensor_map.h"

namespace mr {

// ------------------------------------------------------------------ scales, once per weight

// One 32-bit word (four scales of one weight row) per thread, into the order
// in which the tensor core takes them: for each expert, 128-row tile and
// k-block, words [32 lanes][4 groups of 32 rows] (twice for E2M1: a k-block is
// two words wide).  Tile row i of a gate/up weight is, 16 rows of either in turn,
// gate row or up row of the tile's 64 features.  Scales past the weight's
// edge are zero bytes; they meet zero codes.
//
// Nothing is touched before the kernel launched before has ended: it may be
// the quantiser that writes scale, or a product that still reads packed.  The
// kernel after this one relies on the same wait: its own covers this kernel,
// and so all before.
__global__ void __launch_bounds__(256) mx_pack_kernel(const uint8_t* scale, uint32_t* packed, int64_t words, int R,
                                                      int RT, int KI, int kb, int W, int gate_up) {
    pdl_wait();
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < words; i += (int64_t)gridDim.x * blockDim.x) {
        const int row = (int)(i & 3) * 32 + (int)((i >> 2) & 31);
        int64_t u = i >> 7;
        const int w = (int)(u % W);
        u /= W;
        const int ki = (int)(u % KI);
        u /= KI;
        const int rt = (int)(u % RT);
        const int64_t e = u / RT;
        int r = rt * 128 + row;
        bool in = r < R;
        if (gate_up) {
            const int feature = rt * 64 + (row >> 5) * 16 + (row & 15);
            r = ((row >> 4) & 1) * (R >> 1) + feature;
            in = feature < (R >> 1);
        }
        uint32_t v = 0;
        const uint8_t* s = scale + (e * R + r) * kb;
        for (int b = 0; b < 4; ++b) {
            const int k = (ki * W + w) * 4 + b;
            if (in && k < kb) v |= (uint32_t)s[k] << (8 * b);
        }
        packed[i] = v;
    }
}

cudaError_t launch_mx_pack(const uint8_t* scale, int64_t E, int R, int K, int fp4, int gate_up, void* packed,
                           cudaStream_t st) {
    const ExpertShape s = expert_shape(R, K, fp4, gate_up);
    const int64_t words = E * s.RT * s.KI * s.W * 128;
    int64_t ctas = (words + 255) / 256;
    if (ctas > 152 * 8) ctas = 152 * 8;
    return launch_kernel(mx_pack_kernel, dim3((unsigned)ctas), dim3(256), 0, st, scale, static_cast<uint32_t*>(packed),
                         words, R, s.RT, s.KI, K / 32, s.W, gate_up);
}

// ------------------------------------------------------------------ the combination over a token's experts

// out[m, r] = bf16(add[m, r] + sum_j weights[m, j] y[m * topk + j, r]), j
// ascending in fp32; slots whose id is outside [0, E) are skipped, whatever y
// holds there.  LOW: y and low are the halves of fp32 numbers.  A thread takes
// eight columns of a row (VEC; else one): eight slots' rows are in flight at a
// time.  Bound by reading y: 4096 tokens x 8 x
// 6144 is 403 MB, 72 us (78 % of the peak bandwidth).  Launched so that its
// CTAs are in place when the products end (the wait is for all of them, and
// for the memory they wrote): CTAs of 64 threads find room for their registers
// beside a CTA of the products; of 256 they did not, and started after them
// (one token, rounded rows: 12.0 us for both launches, 12.7 with those).
//
// A launch of its own: added by the products' kernel, tokens finish when the
// last of their experts does, and the CTA that sees it has all their sums to
// do (4096 tokens: 4.0 ms; by panels of columns behind a grid barrier 339-433
// us; the two launches 265).
//
// Lines of y that have been read are given up (discard): nobody reads them
// again, and those that still are in L2 need no way to memory.  Down of 64
// tokens x 8, E2M1, rounded rows: 44.8 us (47.6 without); of 4096, E4M3: 260
// (267).
constexpr int kCombineThreads = 64;
__device__ __forceinline__ void discard_line(const void* line) {
    asm volatile("discard.global.L2 [%0], 128;" ::"l"(line) : "memory");
}
template <bool VEC, bool LOW>
__global__ void __launch_bounds__(kCombineThreads) expert_combine_kernel(const uint16_t* y, const uint16_t* low,
                                                             const int32_t* ids, const float* weights,
                                                             const __nv_bfloat16* add, __nv_bfloat16* out, int64_t M,
                                                             int topk, int R, int E) {
    constexpr int N = VEC ? 8 : 1;
    const bool lines = R % 64 == 0;  // y's rows are whole lines of 128 bytes
    pdl_wait();
    const int per = R / N;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < M * per; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t m = i / per;
        const int r = (int)(i - m * per) * N;
        float s[N];
        auto wide = [](uint4 q, uint4 l, float* f) {  // upper and lower halves of eight numbers
            const uint32_t w[4] = {q.x, q.y, q.z, q.w}, k[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                f[2 * u] = __uint_as_float((w[u] << 16) | (k[u] & 0xFFFFu));
                f[2 * u + 1] = __uint_as_float((w[u] & 0xFFFF0000u) | (k[u] >> 16));
            }
        };
        const uint4 none = make_uint4(0u, 0u, 0u, 0u);
        if (add == nullptr) {
#pragma unroll
            for (int u = 0; u < N; ++u) s[u] = 0.0f;
        } else if (VEC) {
            wide(*reinterpret_cast<const uint4*>(add + m * R + r), none, s);
        } else {
            s[0] = __bfloat162float(add[m * R + r]);
        }
        for (int j0 = 0; j0 < topk; j0 += 8) {
            uint4 v[8], l[8];
            int id[8];
            float w[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                id[u] = -1;
                if (j0 + u >= topk) continue;
                const int64_t f = m * topk + j0 + u, at = f * R + r;
                id[u] = __ldg(ids + f);
                w[u] = __ldg(weights + f);
                if (VEC) v[u] = __ldcg(reinterpret_cast<const uint4*>(y + at));
                else v[u].x = (uint32_t)y[at] << 16;
                if (VEC && LOW) l[u] = __ldcg(reinterpret_cast<const uint4*>(low + at));
                else if (LOW) v[u].x |= low[at];
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if ((unsigned)id[u] >= (unsigned)E) continue;
                float f[8];
                if (VEC) wide(v[u], LOW ? l[u] : none, f);
                else f[0] = __uint_as_float(v[u].x);
#pragma unroll
                for (int q = 0; q < N; ++q) s[q] = __fmaf_rn(w[u], f[q], s[q]);
            }
            if (VEC && lines) {
                // (eight lanes have read a line, all of them or none are here)
                __syncwarp(0xFFu << (threadIdx.x & 24u));
                if ((threadIdx.x & 7) == 0) {
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        if (j0 + u >= topk) continue;
                        discard_line(y + (m * topk + j0 + u) * R + r);
                        if (LOW) discard_line(low + (m * topk + j0 + u) * R + r);
                    }
                }
            }
        }
        if (VEC) {
            uint4 q;
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(q.x) : "f"(s[1]), "f"(s[0]));
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(q.y) : "f"(s[3 % N]), "f"(s[2 % N]));
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(q.z) : "f"(s[5 % N]), "f"(s[4 % N]));
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(q.w) : "f"(s[7 % N]), "f"(s[6 % N]));
            *reinterpret_cast<uint4*>(out + m * R + r) = q;
        } else {
            out[m * R + r] = __float2bfloat16_rn(s[0]);
        }
    }
}

template <bool LOW>
cudaError_t launch_combine(const ExpertCall& c, int sms, cudaStream_t st) {
    const auto* add = static_cast<const __nv_bfloat16*>(c.add);
    auto* out = static_cast<__nv_bfloat16*>(c.out);
    const bool vec = c.R % 8 == 0 && (reinterpret_cast<uintptr_t>(add) | reinterpret_cast<uintptr_t>(out)) % 16 == 0;
    const int64_t work = (int64_t)c.M * (c.R / (vec ? 8 : 1));
    int64_t ctas = (work + kCombineThreads - 1) / kCombineThreads;
    if (ctas > (int64_t)sms * 32) ctas = (int64_t)sms * 32;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kCombineThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const cudaError_t e =
        cudaLaunchKernelEx(&cfg, vec ? expert_combine_kernel<true, LOW> : expert_combine_kernel<false, LOW>,
                           static_cast<const uint16_t*>(c.scratch), static_cast<const uint16_t*>(c.scratch_low),
                           c.topk_ids, c.topk_weights, add, out, (int64_t)c.M, c.topk, c.R, c.E);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// ------------------------------------------------------------------ host

namespace {

bool encode(CUtensorMap* map, const void* ptr, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box) {
    const EncodeTiled fn = encode_tiled();
    if (fn == nullptr) return false;
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, (cuuint32_t)rank, const_cast<void*>(ptr), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool FP4, int OP, bool PAIR, bool SPLIT>
cudaError_t launch_one(const ExpertArgs& a, int grid, cudaStream_t st) {
    static int prepared[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    const auto kernel = expert_kernel<FP4, OP, PAIR, SPLIT>;
    if (!__atomic_load_n(&prepared[dev], __ATOMIC_ACQUIRE)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, ex_smem(OP));
        if (e != cudaSuccess) return e;
        __atomic_store_n(&prepared[dev], 1, __ATOMIC_RELEASE);
    }
    cudaLaunchConfig_t cfg = {};
    const int of = PAIR ? 2 : SPLIT ? a.slices : 1;  // CTAs of a cluster
    cfg.gridDim = dim3((unsigned)(grid / of * of));
    cfg.blockDim = dim3(ex_threads(OP));
    cfg.dynamicSmemBytes = ex_smem(OP);
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    // whatever the launch options: the kernel reads and writes nothing before it has waited for the one before it
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)of;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = PAIR || SPLIT ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, kernel, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}
template <int OP>
cudaError_t launch_op(const ExpertArgs& a, bool fp4, bool pair, int grid, cudaStream_t st) {
    if (a.slices > 1)
        return fp4 ? launch_one<true, OP, false, true>(a, grid, st) : launch_one<false, OP, false, true>(a, grid, st);
    if (fp4) return pair ? launch_one<true, OP, true, false>(a, grid, st) : launch_one<true, OP, false, false>(a, grid, st);
    return pair ? launch_one<false, OP, true, false>(a, grid, st) : launch_one<false, OP, false, false>(a, grid, st);
}

}  // namespace

int launch_expert(const ExpertCall& c, cudaStream_t st, cudaError_t* err) {
    const bool fp4 = c.fp4 != 0;
    const int R = c.R, K = c.K;
    const ExpertShape s = expert_shape(R, K, fp4, c.op == kExGateUp);
    int dev = 0, sms = 0;
    if ((*err = cudaGetDevice(&dev)) != cudaSuccess ||
        (*err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
        return MR_ERR_CUDA;
    ExpertArgs a{};
    const cuuint64_t kbytes = (cuuint64_t)(fp4 ? K / 2 : K);
    {
        const cuuint64_t per = kbytes * (cuuint64_t)R;  // bytes of one expert
        if (c.op == kExGateUp) {
            // [expert][16-row group][gate or up][row of the group][k]: a box of
            // four groups is a tile of 64 features with both of their rows
            const cuuint64_t dims[5] = {kbytes, 16, 2, (cuuint64_t)(R / 32), (cuuint64_t)c.E};
            const cuuint64_t strides[4] = {kbytes, per / 2, 16 * kbytes, per};
            const cuuint32_t box[5] = {128, 16, 2, 4, 1};
            if (!encode(&a.tm_w, c.w, 5, dims, strides, box)) return MR_ERR_UNSUPPORTED;
        } else {
            const cuuint64_t dims[3] = {kbytes, (cuuint64_t)R, (cuuint64_t)c.E};
            const cuuint64_t strides[2] = {kbytes, per};
            const cuuint32_t box[3] = {128, 128, 1};
            if (!encode(&a.tm_w, c.w, 3, dims, strides, box)) return MR_ERR_UNSUPPORTED;
        }
        const cuuint64_t dims[2] = {kbytes, (cuuint64_t)c.x_rows};
        const cuuint64_t strides[1] = {(cuuint64_t)c.ldx};
        const cuuint32_t box[2] = {128, c.gather ? 1u : 16u}, box64[2] = {128, 64};
        if (!encode(&a.tm_x, c.x, 2, dims, strides, box) ||
            (!c.gather && !encode(&a.tm_x64, c.x, 2, dims, strides, box64)))
            return MR_ERR_UNSUPPORTED;
    }
    a.w_scale = c.w_scale;
    a.x_scale = c.x_scale;
    a.x_scale_end = c.x_scale + (c.x_rows - 1) * c.lds + K / 32;
    a.lds = c.lds;
    a.sorted = c.sorted;
    a.experts = c.experts;
    a.out = c.out;
    a.out_scale = c.out_scale;
    a.ldo = c.ldo;
    a.wait_ns = wait_limit_ns();
    a.E = c.E;
    a.R = R;
    a.RT = s.RT;
    a.KI = s.KI;
    a.kb = K / 32;
    a.M = c.M;
    a.topk = c.topk;
    a.mk = c.M * c.topk;
    a.nblk = c.nblk;
    a.block = c.block;
    a.gather = c.gather;
    a.sf_vec = 1;
    for (int v = 8; v <= 16; v *= 2)  // rows whose bytes end on the boundary too: no read past a row
        if (a.kb % v == 0 && c.lds % v == 0 && reinterpret_cast<uintptr_t>(c.x_scale) % v == 0) a.sf_vec = v;
    {  // column tiles: one per expert with rows, and one for every further 256 rows
        const int64_t mk = (int64_t)c.M * c.topk, most = (mk < c.E ? mk : c.E) + mk / kExMaxN + 1;
        a.list_cap = c.op != kExGemm && most <= kExListMax ? (int)most : 0;
    }
    a.out_fmt = c.out_fmt;
    a.flags = launch_flags();
    a.x = c.x;
    a.ldx = c.ldx;
    a.kbytes = (int)kbytes;
    if (c.op == kExDown) a.out = c.scratch, a.out_low = static_cast<uint16_t*>(c.scratch_low);
    const int grid = sms;
    a.slices = expert_slices(a.mk, c.E, s, sms, &a.slice_len);
    const bool pair = a.slices == 1 && expert_pair(a.mk, c.E);
    if (c.op == kExGemm) a.per = expert_gemm_rows(c.M, s.RT, pair, a.slices, sms);
    cudaError_t e = c.op == kExGemm     ? launch_op<kExGemm>(a, fp4, pair, grid, st)
                    : c.op == kExGateUp ? launch_op<kExGateUp>(a, fp4, pair, grid, st)
                                        : launch_op<kExDown>(a, fp4, pair, grid, st);
    if (e == cudaSuccess && c.op == kExDown)
        e = c.scratch_low ? launch_combine<true>(c, sms, st) : launch_combine<false>(c, sms, st);
    *err = e;
    return e == cudaSuccess ? MR_OK : MR_ERR_CUDA;
}

int expert_device_error(int clear) {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_ex_timeout, sizeof(int)) != cudaSuccess) return -1;
    if (clear && v) {
        const int z = 0;
        if (cudaMemcpyToSymbol(g_ex_timeout, &z, sizeof(int)) != cudaSuccess) return -1;
    }
    return v;
}

}  // namespace mr
