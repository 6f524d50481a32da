// The norms around a block of a hybrid model: add_norm (block output into the
// residual stream, and the norm of the sum) and gated_norm (the norm after an
// SSM mixer, fused with its gate).
//
// Both read each input once and write each output once: a row (add_norm) or a
// group of a row's columns (gated_norm) is held by the threads of a block, in FP32, from
// its load through one or two sums of squares to its store: in registers up to 8192
// columns read 8 at a time, or read one by one. What is longer spills, most of a
// thread's share above 8192 columns one by one (0.9 to 2 KB a thread) and above 16384
// 8 at a time (0.2 to 1.1 KB; gated_norm loses up to 0.35 KB from 8192 on). They are
// bound by HBM for many rows (add_norm 6.3 TB/s, gated_norm 5.8) and by latency for few
// (one row of 4096: 2.1 us from a CUDA graph).
#include "overlap.cuh"

namespace rssm {
namespace {

constexpr int kMaxNormDim = 32768;   // columns that the threads of one block hold

struct AddNormArgs {
    const void *u, *x, *gate;
    void *u_out, *n_out;
    const float *w_post, *w;
    int64_t rows, u_stride, x_stride, gate_stride, uo_stride, no_stride;
    int dim;
    float eps, scale, w_off;
};

struct GatedNormArgs {
    const void *y, *z;
    const float* w;
    void* out;
    int64_t rows, y_stride, z_stride, out_stride;
    int group, groups, w_dim;
    int norm_first, act;
    float eps, w_off;
};

// 32 bytes in one access, so that a warp's FP32 accesses have no gaps. L1 is
// passed by for what is read once.
__device__ __forceinline__ void ld32(float (&v)[8], const float* p) {
    asm volatile("ld.global.L1::no_allocate.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]) : "l"(p) : "memory");
}
__device__ __forceinline__ void ld32_keep(float (&v)[8], const float* p) {
    asm("ld.global.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]) : "l"(p));
}
__device__ __forceinline__ void st32(float* p, const float (&v)[8]) {
    asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]) : "memory");
}

// VEC consecutive elements as floats (VEC = 8: aligned to their size, or 1).
template <int VEC>
__device__ __forceinline__ void load_vec(float (&v)[VEC], const float* p) {
    if constexpr (VEC == 8) ld32(v, p);
    else v[0] = *p;
}
template <int VEC>
__device__ __forceinline__ void load_vec(float (&v)[VEC], const __nv_bfloat16* p) {
    if (VEC == 8) {
        const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p));
        const uint32_t r[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[(2 * i) % VEC] = __uint_as_float(r[i] << 16);
            v[(2 * i + 1) % VEC] = __uint_as_float(r[i] & 0xFFFF0000u);
        }
    } else {
        v[0] = __bfloat162float(*p);
    }
}
// Weights stay in cache: every row reads them. p: from past_wait().
template <int VEC>
__device__ __forceinline__ void load_w(float (&v)[VEC], const float* p) {
    if constexpr (VEC == 8) ld32_keep(v, p);
    else asm("ld.global.f32 %0, [%1];" : "=f"(v[0]) : "l"(p));
}
template <int VEC>
__device__ __forceinline__ void store_vec(float* p, const float (&v)[VEC]) {
    if constexpr (VEC == 8) st32(p, v);
    else *p = v[0];
}
template <int VEC>
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float (&v)[VEC]) {
    if (VEC == 8) {
        uint32_t r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[(2 * i) % VEC], v[(2 * i + 1) % VEC]);
            r[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(r[0], r[1], r[2], r[3]);
    } else {
        *p = __float2bfloat16_rn(v[0]);
    }
}

// Sum over the tpr threads that share a row: a power of two of adjacent lanes
// up to 32, else the whole block (a multiple of 32). `slot` alternates between
// two halves of s_red, so consecutive sums need one barrier each.
__device__ __forceinline__ float row_sum(float v, int tpr, float* s_red) {
    if (tpr <= 32) {
        for (int o = tpr >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    }
    v = warp_sum(v);
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = (static_cast<int>(threadIdx.x & 31) < warps) ? s_red[threadIdx.x & 31] : 0.f;
    return warp_sum(t);
}

template <class TU, class TX, int VEC, int VPT>
__global__ void __launch_bounds__(1024) add_norm_kernel(const AddNormArgs a, int tpr) {
    __shared__ float s_red[2][32];
    after_predecessor();
    const int rows_per_block = blockDim.x / tpr;
    const int lane = threadIdx.x % tpr;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * rows_per_block + threadIdx.x / tpr;
    const bool live = row < a.rows;
    const int nvec = a.dim / VEC;
    const float *w_post = past_wait(a.w_post), *w_norm = past_wait(a.w);
    const TU* u = static_cast<const TU*>(a.u) + (live ? row : 0) * a.u_stride;
    const TX* x = static_cast<const TX*>(a.x) + (live ? row : 0) * a.x_stride;
    const TX* gt = static_cast<const TX*>(a.gate) + (live ? row : 0) * a.gate_stride;

    float uv[VPT][VEC], xv[VPT][VEC];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = lane + i * tpr;
        if (live && c < nvec) {
            load_vec<VEC>(uv[i], u + static_cast<int64_t>(c) * VEC);
            if (a.x != nullptr) load_vec<VEC>(xv[i], x + static_cast<int64_t>(c) * VEC);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) uv[i][e] = xv[i][e] = 0.f;
        }
    }
    if (a.x != nullptr) {
        float r = 1.f;
        if (w_post != nullptr) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int e = 0; e < VEC; ++e) ss = fmaf(xv[i][e], xv[i][e], ss);
            r = rsqrtf(row_sum(ss, tpr, s_red[0]) / static_cast<float>(a.dim) + a.eps);
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = lane + i * tpr;
            if (!live || c >= nvec) continue;
            if (w_post != nullptr) {
                float w[VEC];
                load_w<VEC>(w, w_post + c * VEC);
#pragma unroll
                for (int e = 0; e < VEC; ++e) xv[i][e] *= r * (a.w_off + w[e]);
            }
            if (a.gate != nullptr) {
                float g[VEC];
                load_vec<VEC>(g, gt + static_cast<int64_t>(c) * VEC);
#pragma unroll
                for (int e = 0; e < VEC; ++e) xv[i][e] *= g[e];
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) uv[i][e] = fmaf(a.scale, xv[i][e], uv[i][e]);
        }
    }
    if (a.u_out != nullptr) {
        TU* uo = static_cast<TU*>(a.u_out) + (live ? row : 0) * a.uo_stride;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = lane + i * tpr;
            if (live && c < nvec) store_vec<VEC>(uo + static_cast<int64_t>(c) * VEC, uv[i]);
        }
    }
    if (a.n_out == nullptr) return;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) ss = fmaf(uv[i][e], uv[i][e], ss);
    const float r = rsqrtf(row_sum(ss, tpr, s_red[1]) / static_cast<float>(a.dim) + a.eps);
    TX* no = static_cast<TX*>(a.n_out) + (live ? row : 0) * a.no_stride;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = lane + i * tpr;
        if (!live || c >= nvec) continue;
        float w[VEC];
        load_w<VEC>(w, w_norm + c * VEC);
#pragma unroll
        for (int e = 0; e < VEC; ++e) w[e] = uv[i][e] * r * (a.w_off + w[e]);
        store_vec<VEC>(no + static_cast<int64_t>(c) * VEC, w);
    }
}

// act(z). FP32 keeps the exact exponential and division; for BF16 their
// approximations are far inside the rounding and a quarter of the instructions: within
// 2^-20 for |z| <= 8, and, as the rounded product with log2 e grows, within 2^-17 as
// long as the sigmoid is a normal number (z > -87; it is 0 from there on).
template <class T, int ACT>
__device__ __forceinline__ float gate_of(float z) {
    if (sizeof(T) == 4) return (ACT == RSSM_GATE_SILU ? z : 1.f) / (1.f + expf(-z));
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return ACT == RSSM_GATE_SILU ? z * r : r;
}

// VEC elements as they are stored, so that a load can be long under way before
// the values are widened.
template <class T, int VEC>
struct Raw {
    uint32_t w[VEC * sizeof(T) / 4 > 0 ? VEC * sizeof(T) / 4 : 1];
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (VEC == 1) {
            if constexpr (sizeof(T) == 4) w[0] = *reinterpret_cast<const uint32_t*>(p);
            else w[0] = *reinterpret_cast<const uint16_t*>(p);
        } else if constexpr (sizeof(T) == 4) {
            float v[8];
            ld32(v, reinterpret_cast<const float*>(p));
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[i]);
        } else {
            asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(p) : "memory");
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (uint32_t& x : w) x = 0;
    }
    __device__ __forceinline__ void get(float (&v)[VEC]) const {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            if constexpr (sizeof(T) == 4) v[i] = __uint_as_float(w[i]);
            else v[i] = __uint_as_float((i & 1) ? (w[i / 2] & 0xFFFF0000u) : (w[i / 2] << 16));
        }
    }
};

// Short groups are bound by instructions before memory: one group a thread cost 39
// an element and 84 us over 16384 rows of 32 BF16 groups of 128. So a thread takes
// several groups, with the weights of its columns in registers where all groups
// share them (80 us), and loads the next group beside the sums of this one, which
// doubles what is under way at 4 blocks of 256 an SM (69 us, 5.8 TB/s).
template <class T, int VEC, int VPT, int FIRST, int ACT>
__global__ void __launch_bounds__(1024) gated_norm_kernel(const GatedNormArgs a, int tpr, uint32_t items) {
    __shared__ float s_red[2][32];
    after_predecessor();
    const uint32_t per_block = blockDim.x / tpr, step = gridDim.x * per_block;
    const int lane = threadIdx.x % tpr;
    const uint32_t groups = a.groups;
    uint32_t item = blockIdx.x * per_block + threadIdx.x / tpr;
    uint32_t row = item / groups, col = item - row * groups;
    const uint32_t step_row = step / groups, step_col = step - step_row * groups;
    const int nvec = a.group / VEC;
    const bool shared_w = a.w_dim == a.group;
    const float* w_all = past_wait(a.w);
    float wv[VPT][VEC];
    if (shared_w) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = lane + i * tpr;
            if (c >= nvec) continue;
            load_w<VEC>(wv[i], w_all + c * VEC);
#pragma unroll
            for (int e = 0; e < VEC; ++e) wv[i][e] += a.w_off;
        }
    }
    const float inv_n = 1.f / static_cast<float>(a.group);
    int turn = 0;
    Raw<T, VEC> ry[VPT], rz[VPT];
    const auto fetch = [&](uint32_t it, uint32_t r, uint32_t cl) {
        const int64_t at = static_cast<int64_t>(cl) * a.group;
        const T* y = static_cast<const T*>(a.y) + r * a.y_stride + at;
        const T* z = static_cast<const T*>(a.z) + r * a.z_stride + at;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = lane + i * tpr;
            if (it < items && c < nvec) {
                ry[i].load(y + c * VEC);
                rz[i].load(z + c * VEC);
            } else {
                ry[i].clear();
                rz[i].clear();
            }
        }
    };
    fetch(item, row, col);
    // whole blocks go round together: their rows meet at barriers
    for (uint32_t first = blockIdx.x * per_block; first < items; first += step, turn ^= 1) {
        const bool live = item < items;
        const int64_t at = static_cast<int64_t>(col) * a.group;
        T* out = static_cast<T*>(a.out) + row * a.out_stride + at;
        float v[VPT][VEC], g[VPT][VEC];
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            ry[i].get(v[i]);
            rz[i].get(g[i]);
        }
        item += step;
        row += step_row;
        col += step_col;
        if (col >= groups) {
            col -= groups;
            ++row;
        }
        fetch(item, row, col);                 // the next group's loads, beside this one's sums
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                g[i][e] = gate_of<T, ACT>(g[i][e]);
                if (!FIRST) v[i][e] *= g[i][e];
                ss = fmaf(v[i][e], v[i][e], ss);
            }
        const float r = rsqrtf(fmaf(row_sum(ss, tpr, s_red[turn]), inv_n, a.eps));
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = lane + i * tpr;
            if (!live || c >= nvec) continue;
            float w[VEC];
            if (!shared_w) load_w<VEC>(w, w_all + at + c * VEC);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                v[i][e] *= r * (shared_w ? wv[i][e] : a.w_off + w[e]);
                if (FIRST) v[i][e] *= g[i][e];
            }
            store_vec<VEC>(out + c * VEC, v[i]);
        }
    }
}

// Threads per row for nvec vectors of a row, vpt at most per thread: a power of
// two of lanes, or a block of whole warps.
int threads_per_row(int nvec, int vpt) {
    const int need = (nvec + vpt - 1) / vpt;
    if (need > 32) return (need + 31) / 32 * 32;
    int t = 1;
    while (t < need) t *= 2;
    return t;
}

struct NormShape {
    int tpr, vpt, threads;
    int64_t blocks;
};

// vec 8: 1, 2 or 4 vectors a thread; vec 1: 2, 8 or 32 elements. The fewest
// that cover the row with at most 1024 threads: over 16384 rows of 4096 with norms on
// both sides, 1, 2 and 4 vectors a thread took 132, 155 and 175 us (6.2 TB/s at 1),
// over 256 Mamba-2 rows and a single row they did not differ.
NormShape norm_shape(int cols, int vec, int64_t items) {
    const int nvec = cols / vec;
    const int choice[2][3] = {{1, 2, 4}, {2, 8, 32}};
    const int* c = choice[vec == 8 ? 0 : 1];
    NormShape s{};
    for (int i = 0; i < 3; ++i) {
        s.vpt = c[i];
        s.tpr = threads_per_row(nvec, s.vpt);
        if (s.tpr <= 1024) break;
    }
    s.threads = s.tpr <= 32 ? 256 : s.tpr;
    const int per = s.threads / s.tpr;
    s.blocks = (items + per - 1) / per;
    return s;
}

// Whether rows of this type can be read 8 elements at a time.
bool vec_ok(const void* p, int64_t stride, int esz) {
    return (reinterpret_cast<uintptr_t>(p) & (8u * esz - 1)) == 0 && (stride * esz) % (8 * esz) == 0;
}

template <class TU, class TX>
cudaError_t launch_add(const AddNormArgs& a, int vec, const NormShape& s, cudaStream_t st) {
    const dim3 g(static_cast<unsigned>(s.blocks));
    if (vec == 8) {
        if (s.vpt == 1) return launch_overlapped(add_norm_kernel<TU, TX, 8, 1>, g, s.threads, 0, st, a, s.tpr);
        else if (s.vpt == 2) return launch_overlapped(add_norm_kernel<TU, TX, 8, 2>, g, s.threads, 0, st, a, s.tpr);
        else return launch_overlapped(add_norm_kernel<TU, TX, 8, 4>, g, s.threads, 0, st, a, s.tpr);
    } else {
        if (s.vpt == 2) return launch_overlapped(add_norm_kernel<TU, TX, 1, 2>, g, s.threads, 0, st, a, s.tpr);
        else if (s.vpt == 8) return launch_overlapped(add_norm_kernel<TU, TX, 1, 8>, g, s.threads, 0, st, a, s.tpr);
        else return launch_overlapped(add_norm_kernel<TU, TX, 1, 32>, g, s.threads, 0, st, a, s.tpr);
    }
}

template <class T, int FIRST, int ACT>
cudaError_t launch_gated_as(const GatedNormArgs& a, int vec, const NormShape& s, uint32_t items, cudaStream_t st) {
    int sms = 0, smem = 0;
    const cudaError_t e = device_limits(&sms, &smem);
    if (e != cudaSuccess) return e;
    // as many blocks as are resident at 64 registers a thread
    const int64_t most = static_cast<int64_t>(sms) * (1024 / s.threads);
    const dim3 g(static_cast<unsigned>(s.blocks < most ? s.blocks : most));
    if (vec == 8) {
        if (s.vpt == 1) return launch_overlapped(gated_norm_kernel<T, 8, 1, FIRST, ACT>, g, s.threads, 0, st, a, s.tpr, items);
        else if (s.vpt == 2) return launch_overlapped(gated_norm_kernel<T, 8, 2, FIRST, ACT>, g, s.threads, 0, st, a, s.tpr, items);
        else return launch_overlapped(gated_norm_kernel<T, 8, 4, FIRST, ACT>, g, s.threads, 0, st, a, s.tpr, items);
    } else {
        if (s.vpt == 2) return launch_overlapped(gated_norm_kernel<T, 1, 2, FIRST, ACT>, g, s.threads, 0, st, a, s.tpr, items);
        else if (s.vpt == 8) return launch_overlapped(gated_norm_kernel<T, 1, 8, FIRST, ACT>, g, s.threads, 0, st, a, s.tpr, items);
        else return launch_overlapped(gated_norm_kernel<T, 1, 32, FIRST, ACT>, g, s.threads, 0, st, a, s.tpr, items);
    }
}

template <class T>
cudaError_t launch_gated(const GatedNormArgs& a, int vec, const NormShape& s, cudaStream_t st) {
    const uint32_t n = static_cast<uint32_t>(a.rows * a.groups);
    if (a.act == RSSM_GATE_SILU)
        return a.norm_first ? launch_gated_as<T, 1, RSSM_GATE_SILU>(a, vec, s, n, st)
                            : launch_gated_as<T, 0, RSSM_GATE_SILU>(a, vec, s, n, st);
    return a.norm_first ? launch_gated_as<T, 1, RSSM_GATE_SIGMOID>(a, vec, s, n, st)
                        : launch_gated_as<T, 0, RSSM_GATE_SIGMOID>(a, vec, s, n, st);
}

bool float_dtype(int d) { return d == RSSM_F32 || d == RSSM_BF16; }
int elem_size(int d) { return d == RSSM_F32 ? 4 : 2; }

// A row stride: 0 stands for `dim`; otherwise rows must not overlap.
bool row_stride(int64_t s, int dim, int64_t* out) {
    *out = s == 0 ? dim : s;
    return s == 0 || s >= dim;
}

}  // namespace
}  // namespace rssm

using namespace rssm;

extern "C" {

rssm_status rssm_add_norm(const rssm_add_norm_config* c, const void* d_u, const void* d_x, const float* d_w_post,
                          const void* d_gate, const float* d_w, void* d_u_out, void* d_n_out, void* stream) {
    if (c == nullptr || c->rows < 0 || c->rows > 0x7FFFFFFF || c->dim < 1) return RSSM_ERR_INVALID_ARG;
    if (!float_dtype(c->res_dtype) || !float_dtype(c->dtype) || !(c->eps >= 0.f)) return RSSM_ERR_INVALID_ARG;
    if (c->dim > kMaxNormDim) return RSSM_ERR_UNSUPPORTED;
    AddNormArgs a{};
    if (!row_stride(c->u_stride, c->dim, &a.u_stride) || !row_stride(c->x_stride, c->dim, &a.x_stride) ||
        !row_stride(c->u_out_stride, c->dim, &a.uo_stride) || !row_stride(c->n_out_stride, c->dim, &a.no_stride))
        return RSSM_ERR_INVALID_ARG;
    if (c->gate_stride != 0 && c->gate_stride < c->dim) return RSSM_ERR_INVALID_ARG;
    if (c->rows == 0) return RSSM_OK;
    if (d_u == nullptr || (d_u_out == nullptr && d_n_out == nullptr) || (d_n_out != nullptr && d_w == nullptr))
        return RSSM_ERR_INVALID_ARG;
    if (d_x == nullptr && (d_w_post != nullptr || d_gate != nullptr)) return RSSM_ERR_INVALID_ARG;
    a.u = d_u; a.x = d_x; a.gate = d_gate; a.u_out = d_u_out; a.n_out = d_n_out;
    a.w_post = d_w_post; a.w = d_w;
    a.rows = c->rows; a.dim = c->dim; a.gate_stride = c->gate_stride;
    a.eps = c->eps; a.scale = c->scale; a.w_off = c->w_offset;
    const int eu = elem_size(c->res_dtype), ex = elem_size(c->dtype);
    const bool wide = c->dim % 8 == 0 && vec_ok(d_u, a.u_stride, eu) && vec_ok(d_x, a.x_stride, ex) &&
                      vec_ok(d_gate, a.gate_stride, ex) && vec_ok(d_u_out, a.uo_stride, eu) &&
                      vec_ok(d_n_out, a.no_stride, ex) && vec_ok(d_w, 0, 4) && vec_ok(d_w_post, 0, 4);
    const int vec = wide ? 8 : 1;
    const NormShape s = norm_shape(c->dim, vec, c->rows);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (c->res_dtype == RSSM_F32)
        e = c->dtype == RSSM_F32 ? launch_add<float, float>(a, vec, s, st) : launch_add<float, __nv_bfloat16>(a, vec, s, st);
    else
        e = c->dtype == RSSM_F32 ? launch_add<__nv_bfloat16, float>(a, vec, s, st)
                                 : launch_add<__nv_bfloat16, __nv_bfloat16>(a, vec, s, st);
    return e == cudaSuccess ? RSSM_OK : RSSM_ERR_CUDA;
}

rssm_status rssm_gated_norm(const rssm_gated_norm_config* c, const void* d_y, const void* d_z, const float* d_w,
                            void* d_out, void* stream) {
    if (c == nullptr || c->rows < 0 || c->dim < 1 || c->group < 1 || c->dim % c->group != 0) return RSSM_ERR_INVALID_ARG;
    if (c->w_dim != c->dim && c->w_dim != c->group) return RSSM_ERR_INVALID_ARG;
    if (!float_dtype(c->dtype) || !(c->eps >= 0.f)) return RSSM_ERR_INVALID_ARG;
    if (c->act != RSSM_GATE_SILU && c->act != RSSM_GATE_SIGMOID) return RSSM_ERR_INVALID_ARG;
    if (c->norm_first != 0 && c->norm_first != 1) return RSSM_ERR_INVALID_ARG;
    GatedNormArgs a{};
    if (!row_stride(c->y_stride, c->dim, &a.y_stride) || !row_stride(c->z_stride, c->dim, &a.z_stride) ||
        !row_stride(c->out_stride, c->dim, &a.out_stride))
        return RSSM_ERR_INVALID_ARG;
    if (c->rows > 0x7FFFFFFF / (c->dim / c->group)) return RSSM_ERR_INVALID_ARG;
    if (c->group > kMaxNormDim) return RSSM_ERR_UNSUPPORTED;
    if (c->rows == 0) return RSSM_OK;
    if (d_y == nullptr || d_z == nullptr || d_w == nullptr || d_out == nullptr) return RSSM_ERR_INVALID_ARG;
    a.y = d_y; a.z = d_z; a.w = d_w; a.out = d_out;
    a.rows = c->rows; a.group = c->group; a.groups = c->dim / c->group; a.w_dim = c->w_dim;
    a.norm_first = c->norm_first; a.act = c->act; a.eps = c->eps; a.w_off = c->w_offset;
    const int es = elem_size(c->dtype);
    const bool wide = c->group % 8 == 0 && vec_ok(d_y, a.y_stride, es) && vec_ok(d_z, a.z_stride, es) &&
                      vec_ok(d_out, a.out_stride, es) && vec_ok(d_w, 0, 4);
    const int vec = wide ? 8 : 1;
    const NormShape s = norm_shape(c->group, vec, a.rows * a.groups);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = c->dtype == RSSM_F32 ? launch_gated<float>(a, vec, s, st)
                                               : launch_gated<__nv_bfloat16>(a, vec, s, st);
    return e == cudaSuccess ? RSSM_OK : RSSM_ERR_CUDA;
}

}  // extern "C"
