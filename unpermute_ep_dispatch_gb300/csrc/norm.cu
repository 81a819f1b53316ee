// norm.cu -- layer norm and its root-mean-square form (ep_layer_norm), and their gradients
// (ep_layer_norm_backward).
//
//   s = x + residual,  mean = sum s / H,  rstd = (sum (s - mean)^2 / H + eps)^-1/2   (mean 0 for RMS)
//   y = (s - mean) rstd weight + bias
//   g = dy weight,  xh = (x - mean) rstd
//   dx = rstd (g - sum g / H - xh sum(g xh) / H) + grad_sum      (RMS: without sum g)
//   dweight = sum over rows of dy xh,  dbias = sum over rows of dy
//
// Bound by HBM: every row is read once and written once. A block owns a row, a thread 8, 16 or 32 of
// its columns in chunks of 16 bytes, and blocks walk over the rows with the row kept in registers
// between the sums and the output. Each thread copies its own chunks of the rows to come into its own
// slots of shared memory (cp.async, two or four rows ahead): no barrier and no wait but the thread's
// own, and one block a multiprocessor keeps 40 KB or more on the way. 8192 x 7168 bf16 rows with a
// residual in and out take 72.4 us into bf16 (470 MB: 70 at a copy's rate), 73 into e4m3 (62) and 81.5 into
// both (79), 4097 x 4096 fp32 rows 16.8 (15); the gradient of 8192 x 7168 bf16 rows, joined, 82 (470 MB: 70),
// of 4096 x 7168 fp32 65 (62).
//
// The weights' gradients: a thread keeps the sums of its columns over all of its block's rows in
// registers; the blocks' sums go to the workspace and a second kernel adds them in a fixed order.
#include <cuda_fp8.h>

#include "epd_math.cuh"

namespace epd {
namespace {

constexpr int kMaxHidden = 16384;
constexpr int kNormThreads = 512;
constexpr int kNormMaxSms = 160;    // blocks that the workspace has room for, per block of a multiprocessor
constexpr int kReduceThreads = 256;
constexpr int kRingBytes = 224 * 1024;  // of the 227 KB that a multiprocessor's blocks share
constexpr size_t kAheadBytes = 56 * 1024;
constexpr unsigned kAll = 0xffffffffu;

struct NormArgs {
    const uint8_t *x, *residual;
    const float *weight, *bias;
    int T, chunks, rms, stages;  // chunks: 16-byte pieces of a row
    float eps, inv_h;
    uint8_t *sum, *y, *yq;
    float *yscale, *mean, *rstd;
};

struct NormGradArgs {
    const uint8_t *dy, *x, *grad_sum;
    const float *weight, *mean, *rstd;
    int T, chunks, rms, stages;
    float inv_h;
    uint8_t *dx;
    float *dweight, *dbias;  // the sums themselves (one block) or the workspace's [block][2][H]
    int64_t block_stride;    // floats between two blocks' sums
};

template <int BYTES>
__device__ __forceinline__ void copy_piece(uint32_t dst_smem, const void *src) {
    if (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst_smem), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst_smem), "l"(src), "n"(BYTES) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t p) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t p) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(p) : "memory");
    return v;
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until the oldest of `stages` groups has landed.
__device__ __forceinline__ void copy_wait(int stages) {
    if (stages == 4) asm volatile("cp.async.wait_group 3;" ::: "memory");
    else if (stages == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Sums of a and b over the block's warps (16 at most), in every thread. The two take one exchange to
// lie in a half-warp each and go on together. `part` alternates between two calls, so that one barrier a
// call is enough.
__device__ __forceinline__ void block_add(float &a, float &b, float (&part)[2][16]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const bool upper = lane & 16;
    float v = (upper ? b : a) + __shfl_xor_sync(kAll, upper ? a : b, 16);
#pragma unroll
    for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    if (warps > 1) {
        if ((lane & 15) == 0) part[lane >> 4][warp] = v;
        __syncthreads();
        v = (lane & 15) < warps ? part[lane >> 4][lane & 15] : 0.0f;
#pragma unroll
        for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    }
    a = __shfl_sync(kAll, v, 0);
    b = __shfl_sync(kAll, v, 16);
}

// The same of one sum.
__device__ __forceinline__ void block_add(float &a, float (&part)[16]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int o = 16; o; o >>= 1) a += __shfl_xor_sync(kAll, a, o);
    if (warps == 1) return;
    if (lane == 0) part[warp] = a;
    __syncthreads();
    a = (lane & 15) < warps ? part[lane & 15] : 0.0f;
#pragma unroll
    for (int o = 8; o; o >>= 1) a += __shfl_xor_sync(kAll, a, o);
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// x^-1/2 to a unit in the last place: the hardware's, 2 units off, and a step of Newton's. It is on every
// row's way from its sums to its output, where a root and a division take three times as long.
__device__ __forceinline__ float inverse_root(float x) {
    const float r = rsqrtf(x);
    const float d = fmaf(-x * r, r, 1.0f);  // (NaN of 0 and of infinity, whose root is exact)
    return d < 1.0f ? fmaf(0.5f * r, d, r) : r;
}

// A chunk in 32 bits, two columns to an instruction: the C columns of 16 bytes of T, so that a warp's
// loads and stores of x are 512 bytes in a row.
template <int C>
struct Columns {
    float2 v[C / 2];
};

template <int C>
__device__ __forceinline__ void unpack_bf16(uint32_t p, Columns<C> &f) {
    uint32_t u[C / 2];
    if constexpr (C == 8) {
        const uint4 x = lds16(p);
        u[0] = x.x, u[1] = x.y, u[2] = x.z, u[3] = x.w;
    } else {
        const uint2 x = lds8(p);
        u[0] = x.x, u[1] = x.y;
    }
#pragma unroll
    for (int j = 0; j < C / 2; ++j) f.v[j] = make_float2(lo_bf16(u[j]), hi_bf16(u[j]));
}
template <int C>
__device__ __forceinline__ void store_bf16(uint8_t *p, const Columns<C> &f) {
    if constexpr (C == 8)
        st16(p, make_uint4(pack2_bf16(f.v[0].x, f.v[0].y), pack2_bf16(f.v[1].x, f.v[1].y), pack2_bf16(f.v[2].x, f.v[2].y), pack2_bf16(f.v[3].x, f.v[3].y)));
    else
        *reinterpret_cast<uint2 *>(p) = make_uint2(pack2_bf16(f.v[0].x, f.v[0].y), pack2_bf16(f.v[1].x, f.v[1].y));
}

template <typename T>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16> {
    static constexpr int C = 8;
    static __device__ __forceinline__ void unpack(uint32_t p, Columns<8> &f) { unpack_bf16(p, f); }
    static __device__ __forceinline__ void store(uint8_t *p, const Columns<8> &f) { store_bf16(p, f); }
};
template <>
struct Chunk<float> {
    static constexpr int C = 4;
    static __device__ __forceinline__ void unpack(uint32_t p, Columns<4> &f) {
        const uint4 w = lds16(p);
        f.v[0] = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
        f.v[1] = make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
    }
    static __device__ __forceinline__ void store(uint8_t *p, const Columns<4> &f) {
        st16(p, make_uint4(__float_as_uint(f.v[0].x), __float_as_uint(f.v[0].y), __float_as_uint(f.v[1].x), __float_as_uint(f.v[1].y)));
    }
};

// Starts the copy of this thread's chunks of a row, BYTES each, into its slots of `at` (chunk i of
// thread t at (i * blockDim.x + t) * BYTES).
template <int BYTES, int NV>
__device__ __forceinline__ void fetch_row(uint32_t at, const uint8_t *src, int64_t row, int chunks) {
    const int n = blockDim.x, tid = threadIdx.x;
    const uint8_t *p = src + (row * chunks + tid) * BYTES;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (tid + i * n < chunks) copy_piece<BYTES>(at + (i * n + tid) * BYTES, p + i * n * BYTES);
}

template <int C>
__device__ __forceinline__ void load_floats(const float *p, int c, Columns<C> &f, float none) {
#pragma unroll
    for (int j = 0; j < C / 2; ++j) f.v[j] = p ? __ldg(reinterpret_cast<const float2 *>(p + C * (int64_t)c) + j) : both(none);
}

template <typename T, int NV>
__global__ void __launch_bounds__(kNormThreads, NV * Chunk<T>::C <= 8 ? 2 : 1) norm_kernel(NormArgs a) {
    constexpr int C = Chunk<T>::C;
    constexpr int KEEP = NV * C <= 16 ? NV : 1;  // chunks whose weights stay in registers
    extern __shared__ uint4 s_dyn[];
    const uint32_t s_ring = smem_addr(s_dyn);
    __shared__ float s_part[3][2][16];
    const int tid = threadIdx.x, n = blockDim.x;
    const int stage = (a.residual ? 2 : 1) * NV * n * 16;
    pdl_wait();
    pdl_trigger();
    auto fetch = [&](int64_t row, int s) {
        if (row < a.T) {
            fetch_row<16, NV>(s_ring + s * stage, a.x, row, a.chunks);
            if (a.residual) fetch_row<16, NV>(s_ring + s * stage + NV * n * 16, a.residual, row, a.chunks);
        }
        copy_commit();
    };
    for (int s = 0; s < a.stages; ++s) fetch(blockIdx.x + (int64_t)s * gridDim.x, s);
    Columns<C> w[KEEP], b[KEEP];
    auto load_weights = [&](int i, int k) {
        if (tid + i * n >= a.chunks) return;
        load_floats(a.weight, tid + i * n, w[k], 1.0f);
        load_floats(a.bias, tid + i * n, b[k], 0.0f);
    };
    if (KEEP == NV) {
#pragma unroll
        for (int i = 0; i < KEEP; ++i) load_weights(i, i);
    }
    int s = 0, turn = 0;
    for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
        copy_wait(a.stages);
        Columns<C> v[NV];
        float2 sum2 = both(0.0f), sq2 = both(0.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = tid + i * n;
            if (c >= a.chunks) continue;
            const uint32_t slot = s_ring + s * stage + c * 16;
            Chunk<T>::unpack(slot, v[i]);
            if (a.residual) {
                Columns<C> r;
                Chunk<T>::unpack(slot + NV * n * 16, r);
#pragma unroll
                for (int j = 0; j < C / 2; ++j) v[i].v[j] = __fadd2_rn(v[i].v[j], r.v[j]);
                if (a.sum) Chunk<T>::store(a.sum + (row * a.chunks + c) * 16, v[i]);
            }
#pragma unroll
            for (int j = 0; j < C / 2; ++j) {
                sum2 = __fadd2_rn(sum2, v[i].v[j]);
                sq2 = __ffma2_rn(v[i].v[j], v[i].v[j], sq2);
            }
        }
        float mean = 0.0f, sq = sq2.x + sq2.y, var;
        if (a.rms) {
            block_add(sq, s_part[turn][0]);
            var = sq * a.inv_h;
        } else {
            mean = sum2.x + sum2.y;
            block_add(mean, sq, s_part[turn]);
            mean = __fdiv_rn(mean, (float)(a.chunks * C));
            var = fmaf(-mean, mean, sq * a.inv_h);
            // The squares' mean less the mean's square loses a bit at most where the mean is below the
            // deviation; for the rows where it is not, and those whose squares do not fit, the centred values are
            // summed.
            if (mean * mean > var || var == INFINITY) {
                sq2 = both(0.0f);
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (tid + i * n < a.chunks) {
#pragma unroll
                        for (int j = 0; j < C / 2; ++j) {
                            const float2 d = __fadd2_rn(v[i].v[j], both(-mean));
                            sq2 = __ffma2_rn(d, d, sq2);
                        }
                    }
                sq = sq2.x + sq2.y;
                block_add(sq, s_part[2][0]);
                var = sq * a.inv_h;
            }
        }
        turn ^= 1;
        const float rstd = inverse_root(var + a.eps);
        fetch(row + (int64_t)a.stages * gridDim.x, s);
        if (++s == a.stages) s = 0;
        if (tid == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
        auto scaled = [&](int i) {
            const int k = KEEP == NV ? i : 0;
            if (KEEP != NV) load_weights(i, 0);
            Columns<C> o;
#pragma unroll
            for (int j = 0; j < C / 2; ++j) o.v[j] = __ffma2_rn(__fmul2_rn(__fadd2_rn(v[i].v[j], both(-mean)), both(rstd)), w[k].v[j], b[k].v[j]);
            if (a.y) store_bf16(a.y + (row * a.chunks + tid + i * n) * (2 * C), o);
            return o;
        };
        if (!a.yq) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (tid + i * n < a.chunks) scaled(i);
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (tid + i * n < a.chunks) v[i] = scaled(i);
            // 128 columns are G neighbouring lanes, all of them with a chunk or none. The largest of a thread's
            // chunks take their exchanges together: after each of the first ones a lane has half as many, and
            // in the end the one of chunk `mine`, whose scale it finds for all of them (8192 x 4096 fp32 into
            // e4m3 41 us; 55 with an exchange and two divisions for every chunk). The quotients' remainders, which
            // make them the rounded ones, take 2 to 4 us of that size's and the next's (42.3; 8192 x 8192 bf16 68.5).
            constexpr int G = 128 / C;
            const int lane = tid & 31;
            float top[NV];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                top[i] = 0.0f;
                if (tid + i * n >= a.chunks) continue;
#pragma unroll
                for (int j = 0; j < C / 2; ++j) top[i] = fmaxf(top[i], fmaxf(fabsf(v[i].v[j].x), fabsf(v[i].v[j].y)));
            }
            int mine = 0;
#pragma unroll
            for (int step = 1, d = G / 2; d; step *= 2, d /= 2) {
                if (step < NV) {
                    const bool upper = lane & d;
                    mine += upper ? step : 0;
#pragma unroll
                    for (int i = 0; i < NV / (2 * step); ++i) {
                        const float other = __shfl_xor_sync(kAll, upper ? top[2 * i] : top[2 * i + 1], d);
                        top[i] = fmaxf(upper ? top[2 * i + 1] : top[2 * i], other);
                    }
                } else {
                    top[0] = fmaxf(top[0], __shfl_xor_sync(kAll, top[0], d));
                }
            }
            const float scale = e4m3_scale(top[0]), inv = __fdiv_rn(1.0f, scale);
            const int group = (tid + mine * n) / G;
            if ((lane & (G / NV - 1)) == 0 && group * G < a.chunks) a.yscale[row * (a.chunks / G) + group] = scale;
            const bool tiny = __any_sync(kAll, scale < kTinyScale);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = tid + i * n;
                int from = lane & ~(G - 1);
#pragma unroll
                for (int step = 1, d = G / 2; step < NV; step *= 2, d /= 2) from += i & step ? d : 0;
                const float by = __shfl_sync(kAll, scale, from), inverse = __shfl_sync(kAll, inv, from);
                if (c >= a.chunks) continue;
                float f[C];
                if (tiny) {
#pragma unroll
                    for (int j = 0; j < C; ++j) f[j] = j & 1 ? v[i].v[j / 2].y : v[i].v[j / 2].x;
                    divide_all(f, by);
                } else {
                    const Quotient quotient(by, inverse);
#pragma unroll
                    for (int j = 0; j < C; j += 2) {
                        const float2 u = quotient(v[i].v[j / 2]);
                        f[j] = u.x, f[j + 1] = u.y;
                    }
                }
                uint32_t q[C / 4];
#pragma unroll
                for (int j = 0; j < C / 4; ++j)
                    q[j] = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * j], f[4 * j + 1]), __NV_SATFINITE, __NV_E4M3) |
                           (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(f[4 * j + 2], f[4 * j + 3]), __NV_SATFINITE, __NV_E4M3) << 16;
                uint8_t *const out = a.yq + (row * a.chunks + c) * C;
                if constexpr (C == 8) *reinterpret_cast<uint2 *>(out) = make_uint2(q[0], q[1]);
                else *reinterpret_cast<uint32_t *>(out) = q[0];
            }
        }
    }
}

template <typename T, int NV>
__global__ void __launch_bounds__(kNormThreads) norm_backward_kernel(NormGradArgs a) {
    constexpr int C = Chunk<T>::C;
    constexpr int KEEP = NV * C <= 16 ? NV : 1;
    extern __shared__ uint4 s_dyn[];
    const uint32_t s_ring = smem_addr(s_dyn);
    __shared__ float s_part[2][2][16];
    // every warp has a row's rstd and mean copied for itself (as plain loads a row ahead the compiler
    // put them where their latency showed: 8192 x 7168 took 111 us)
    __shared__ uint2 s_statistics[4][16];
    const int tid = threadIdx.x, n = blockDim.x;
    const uint32_t statistics = smem_addr(&s_statistics[0][tid >> 5]);
    // a stage: x, grad_sum (if any), dy
    const int dy_off = (a.grad_sum ? 2 : 1) * NV * n * 16, stage = dy_off + NV * n * (2 * C);
    pdl_wait();
    pdl_trigger();
    auto fetch = [&](int64_t row, int s) {
        if (row < a.T) {
            const uint32_t at = s_ring + s * stage;
            fetch_row<16, NV>(at, a.x, row, a.chunks);
            if (a.grad_sum) fetch_row<16, NV>(at + NV * n * 16, a.grad_sum, row, a.chunks);
            fetch_row<2 * C, NV>(at + dy_off, a.dy, row, a.chunks);
            const int lane = tid & 31;
            if (lane < (a.rms ? 1 : 2)) copy_piece<4>(statistics + s * (16 * 8) + lane * 4, (lane ? a.mean : a.rstd) + row);
        }
        copy_commit();
    };
    for (int s = 0; s < a.stages; ++s) fetch(blockIdx.x + (int64_t)s * gridDim.x, s);
    Columns<C> w[KEEP], dw[NV] = {}, db[NV] = {};
    if (KEEP == NV) {
#pragma unroll
        for (int i = 0; i < KEEP; ++i)
            if (tid + i * n < a.chunks) load_floats(a.weight, tid + i * n, w[i], 1.0f);
    }
    int s = 0, turn = 0;
    for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
        copy_wait(a.stages);
        __syncwarp();  // the statistics are the warp's
        const uint32_t at = s_ring + s * stage;
        const uint2 st = lds8(statistics + s * (16 * 8));
        const float rstd = __uint_as_float(st.x), mean = a.rms ? 0.0f : __uint_as_float(st.y);
        auto read = [&](int c, Columns<C> &dy, Columns<C> &xh) {
            unpack_bf16(at + dy_off + c * (2 * C), dy);
            Chunk<T>::unpack(at + c * 16, xh);
#pragma unroll
            for (int j = 0; j < C / 2; ++j) xh.v[j] = __fmul2_rn(__fadd2_rn(xh.v[j], both(-mean)), both(rstd));
        };
        // a wide row's chunks are unpacked again for the second pass: they would not stay in registers
        Columns<C> g[KEEP], xh[KEEP];
        float2 sg2 = both(0.0f), sgx2 = both(0.0f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = tid + i * n;
            if (c >= a.chunks) continue;
            const int k = KEEP == NV ? i : 0;
            if (KEEP != NV) load_floats(a.weight, c, w[k], 1.0f);
            read(c, g[k], xh[k]);
#pragma unroll
            for (int j = 0; j < C / 2; ++j) {
                dw[i].v[j] = __ffma2_rn(g[k].v[j], xh[k].v[j], dw[i].v[j]);
                db[i].v[j] = __fadd2_rn(db[i].v[j], g[k].v[j]);
                g[k].v[j] = __fmul2_rn(g[k].v[j], w[k].v[j]);
                sg2 = __fadd2_rn(sg2, g[k].v[j]);
                sgx2 = __ffma2_rn(g[k].v[j], xh[k].v[j], sgx2);
            }
        }
        float sg = sg2.x + sg2.y, sgx = sgx2.x + sgx2.y;
        block_add(sg, sgx, s_part[turn]);
        turn ^= 1;
        // dx = g rstd - xh (rstd sgx / H) - rstd sg / H
        const float by_x = -rstd * (sgx * a.inv_h), by_1 = a.rms ? 0.0f : -rstd * (sg * a.inv_h);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = tid + i * n;
            if (c >= a.chunks) continue;
            const int k = KEEP == NV ? i : 0;
            if (KEEP != NV) {
                load_floats(a.weight, c, w[k], 1.0f);
                read(c, g[k], xh[k]);
#pragma unroll
                for (int j = 0; j < C / 2; ++j) g[k].v[j] = __fmul2_rn(g[k].v[j], w[k].v[j]);
            }
            Columns<C> o;
#pragma unroll
            for (int j = 0; j < C / 2; ++j)
                o.v[j] = __ffma2_rn(xh[k].v[j], both(by_x), __ffma2_rn(g[k].v[j], both(rstd), both(by_1)));
            if (a.grad_sum) {
                Columns<C> r;
                Chunk<T>::unpack(at + NV * n * 16 + c * 16, r);
#pragma unroll
                for (int j = 0; j < C / 2; ++j) o.v[j] = __fadd2_rn(o.v[j], r.v[j]);
            }
            Chunk<T>::store(a.dx + (row * a.chunks + c) * 16, o);
        }
        fetch(row + (int64_t)a.stages * gridDim.x, s);
        if (++s == a.stages) s = 0;
    }
    float *const outs[2] = {a.dweight, a.dbias};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (!outs[k]) continue;
        float *const out = outs[k] + blockIdx.x * a.block_stride;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = tid + i * n;
            if (c >= a.chunks) continue;
#pragma unroll
            for (int j = 0; j < C / 4; ++j) {
                const float2 p = k ? db[i].v[2 * j] : dw[i].v[2 * j], q = k ? db[i].v[2 * j + 1] : dw[i].v[2 * j + 1];
                *reinterpret_cast<float4 *>(out + C * (int64_t)c + 4 * j) = make_float4(p.x, p.y, q.x, q.y);
            }
        }
    }
}

// out[h] = sum over blocks of part[block][h]: a block takes 32 columns, its 32 groups of eight lanes
// every 32nd of the rows, joined in the groups' order. blockIdx.y chooses the weight's or the bias's.
__global__ void __launch_bounds__(kReduceThreads) norm_reduce_kernel(const float *part, int blocks, int64_t stride, int H,
                                                                     float *dweight, float *dbias) {
    __shared__ float4 s_sum[kReduceThreads / 32][8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const bool second = blockIdx.y == 1 || !dweight;
    float *const out = second ? dbias : dweight;
    const float *const in = part + (second ? H : 0);
    const int h = (blockIdx.x * 8 + (lane & 7)) * 4;
    pdl_wait();
    pdl_trigger();
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (h < H) {
#pragma unroll 8
        for (int b = warp * 4 + (lane >> 3); b < blocks; b += kReduceThreads / 8) {
            const float4 p = __ldcg(reinterpret_cast<const float4 *>(in + b * stride + h));
            v.x += p.x, v.y += p.y, v.z += p.z, v.w += p.w;
        }
    }
#pragma unroll
    for (int o = 8; o < 32; o <<= 1) {
        v.x += __shfl_xor_sync(kAll, v.x, o), v.y += __shfl_xor_sync(kAll, v.y, o);
        v.z += __shfl_xor_sync(kAll, v.z, o), v.w += __shfl_xor_sync(kAll, v.w, o);
    }
    if (lane < 8) s_sum[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && lane < 8 && h < H) {
#pragma unroll
        for (int i = 1; i < kReduceThreads / 32; ++i) {
            const float4 p = s_sum[i][lane];
            v.x += p.x, v.y += p.y, v.z += p.z, v.w += p.w;
        }
        *reinterpret_cast<float4 *>(out + h) = v;
    }
}

// Columns of a thread, threads of a block (a multiple of 32) and blocks of a multiprocessor: 8 columns
// where that is a warp or two, 16 up to 512 threads (the sums over the block and the loop cost
// every warp the same, whatever it holds: 8192 x 2048 bf16 with 8 took 20.8 us, with 16 15.0), else 32.
struct NormShape {
    int columns, threads, per_sm;
};
inline NormShape norm_shape(int H) {
    NormShape s;
    s.columns = H <= 512 ? 8 : H <= 16 * kNormThreads ? 16 : 32;
    s.threads = ((H + s.columns - 1) / s.columns + 31) / 32 * 32;
    s.per_sm = kNormThreads / s.threads;  // by the kernels' registers
    return s;
}

inline int norm_max_blocks(int H) { return kNormMaxSms * norm_shape(H).per_sm; }

// Rows ahead: four while a multiprocessor's blocks have 56 KB of them on the way, else two, or one where two
// do not fit. More only make the multiprocessors' shares of the memory uneven: 8192 x 7168 bf16 with a
// residual into bf16 81.5 us with four rows (112 KB) ahead and 72.4 with two, into both 91 and 81.5; 4097 x
// 4096 fp32 17.2 and 16.8 (but 8192 x 2048, which L2 holds, 19.0 and 20.6).
inline int norm_stages(size_t stage_bytes, int per_sm) {
    const size_t room = (size_t)kRingBytes / per_sm - 2048;
    return 4 * stage_bytes <= room && 4 * stage_bytes * per_sm <= kAheadBytes ? 4 : 2 * stage_bytes <= room ? 2 : 1;
}

template <auto kernel, typename A>
epd_status_t launch_rows(A a, const NormShape &s, int grid, size_t stage_bytes, cudaStream_t st) {
    a.stages = norm_stages(stage_bytes, s.per_sm);
    if (const epd_status_t rc = allow_smem<kernel>(kRingBytes)) return rc;
    return launch_pdl(kernel, grid, s.threads, a.stages * stage_bytes, st, a);
}

bool floats_ok(const float *p) { return aligned16(p); }  // read and written 16 bytes at a time

}  // namespace
}  // namespace epd

extern "C" epd_status_t ep_layer_norm(const void *x, epd_dtype_t dtype, const void *residual, const float *weight,
                                      const float *bias, int num_tokens, int hidden, float eps, epd_norm_t kind,
                                      void *sum, void *y, void *y_q, float *y_scale, float *mean, float *rstd,
                                      epd_stream_t stream) {
    using namespace epd;
    const int T = num_tokens, H = hidden;
    if (dtype != EPD_F32 && dtype != EPD_BF16) return EPD_ERR_INVALID_ARG;
    if (kind != EPD_NORM_LAYER && kind != EPD_NORM_RMS) return EPD_ERR_INVALID_ARG;
    if (T < 0 || H < 8 || H % 8 != 0 || !(eps >= 0.0f)) return EPD_ERR_INVALID_ARG;
    if ((y_q != nullptr) != (y_scale != nullptr) || (y_q && H % 128 != 0)) return EPD_ERR_INVALID_ARG;
    if (sum && !residual) return EPD_ERR_INVALID_ARG;
    if (H > kMaxHidden) return EPD_ERR_UNSUPPORTED;
    if (T == 0) return EPD_OK;
    if (!x || (!y && !y_q)) return EPD_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(residual) || !aligned16(sum) || !aligned16(y) || !aligned8(y_q) ||
        !floats_ok(weight) || !floats_ok(bias) || !aligned4(y_scale) || !aligned4(mean) || !aligned4(rstd))
        return EPD_ERR_INVALID_ARG;
    NormArgs a;
    a.x = static_cast<const uint8_t *>(x);
    a.residual = static_cast<const uint8_t *>(residual);
    a.weight = weight;
    a.bias = bias;
    a.T = T;
    a.chunks = H / (dtype == EPD_F32 ? 4 : 8);
    a.rms = kind == EPD_NORM_RMS;
    a.eps = eps;
    a.inv_h = 1.0f / (float)H;
    a.sum = static_cast<uint8_t *>(sum);
    a.y = static_cast<uint8_t *>(y);
    a.yq = static_cast<uint8_t *>(y_q);
    a.yscale = y_scale;
    a.mean = mean;
    a.rstd = rstd;
    NormShape s = norm_shape(H);
    // Eight columns leave room in the registers for twice the blocks (16384 x 512 bf16 into e4m3 11.7 us, 2.4 more
    // with as many as of 16 columns, which spill in half the registers: 8192 x 7168 72 -> 92).
    if (s.columns == 8) s.per_sm *= 2;
    const int most = sm_count() * s.per_sm, grid = T < most ? T : most;
    const size_t stage = (size_t)(residual ? 2 : 1) * s.threads * s.columns * (dtype == EPD_F32 ? 4 : 2);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == EPD_F32)
        return s.columns == 8    ? launch_rows<norm_kernel<float, 2>>(a, s, grid, stage, st)
               : s.columns == 16 ? launch_rows<norm_kernel<float, 4>>(a, s, grid, stage, st)
                                 : launch_rows<norm_kernel<float, 8>>(a, s, grid, stage, st);
    return s.columns == 8    ? launch_rows<norm_kernel<__nv_bfloat16, 1>>(a, s, grid, stage, st)
           : s.columns == 16 ? launch_rows<norm_kernel<__nv_bfloat16, 2>>(a, s, grid, stage, st)
                             : launch_rows<norm_kernel<__nv_bfloat16, 4>>(a, s, grid, stage, st);
}

extern "C" size_t epd_norm_workspace_bytes(int hidden) {
    if (hidden < 8 || hidden % 8 != 0 || hidden > epd::kMaxHidden) return 0;
    return (size_t)epd::norm_max_blocks(hidden) * 2 * hidden * 4;
}

extern "C" epd_status_t ep_layer_norm_backward(const void *dy, const void *x, epd_dtype_t dtype, const float *weight,
                                               const float *mean, const float *rstd, const void *grad_sum,
                                               int num_tokens, int hidden, epd_norm_t kind, void *workspace, void *dx,
                                               float *dweight, float *dbias, epd_stream_t stream) {
    using namespace epd;
    const int T = num_tokens, H = hidden;
    if (dtype != EPD_F32 && dtype != EPD_BF16) return EPD_ERR_INVALID_ARG;
    if (kind != EPD_NORM_LAYER && kind != EPD_NORM_RMS) return EPD_ERR_INVALID_ARG;
    if (T < 0 || H < 8 || H % 8 != 0) return EPD_ERR_INVALID_ARG;
    if (H > kMaxHidden) return EPD_ERR_UNSUPPORTED;
    if (T > 0 && (!dy || !x || !rstd || !dx || (kind == EPD_NORM_LAYER && !mean))) return EPD_ERR_INVALID_ARG;
    if (!aligned16(dy) || !aligned16(x) || !aligned16(grad_sum) || !aligned16(dx) || !floats_ok(weight) ||
        !floats_ok(dweight) || !floats_ok(dbias) || !aligned4(mean) || !aligned4(rstd) || !aligned16(workspace))
        return EPD_ERR_INVALID_ARG;
    const bool sums = dweight || dbias;
    if (sums && !workspace) return EPD_ERR_INVALID_ARG;
    if (T == 0 && !sums) return EPD_OK;
    const NormShape s = norm_shape(H);
    const int sms = sm_count() < kNormMaxSms ? sm_count() : kNormMaxSms;
    // Past two blocks a multiprocessor, four rows a block at least: what the blocks sum up is added
    // afterwards (4096 x 128: 2432 blocks 12.3 us, 1024 7.2; 333 x 1032: 304 blocks 5.4 us, 84 6.0).
    const int most = sms * s.per_sm, quarter = (T + 3) / 4, few = T < 2 * sms ? T : 2 * sms;
    const int want = !sums ? T : quarter > few ? quarter : few, grid = want < 1 ? 1 : want < most ? want : most;
    NormGradArgs a;
    a.dy = static_cast<const uint8_t *>(dy);
    a.x = static_cast<const uint8_t *>(x);
    a.grad_sum = static_cast<const uint8_t *>(grad_sum);
    a.weight = weight;
    a.mean = mean;
    a.rstd = rstd;
    a.T = T;
    a.chunks = H / (dtype == EPD_F32 ? 4 : 8);
    a.rms = kind == EPD_NORM_RMS;
    a.inv_h = 1.0f / (float)H;
    a.dx = static_cast<uint8_t *>(dx);
    float *const part = static_cast<float *>(workspace);
    // one block's sums are the gradients themselves
    a.block_stride = grid == 1 ? 0 : 2 * (int64_t)H;
    a.dweight = !dweight ? nullptr : grid == 1 ? dweight : part;
    a.dbias = !dbias ? nullptr : grid == 1 ? dbias : part + H;
    const size_t stage = (size_t)s.threads * s.columns * (2 + (grad_sum ? 2 : 1) * (dtype == EPD_F32 ? 4 : 2));
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    epd_status_t rc;
    if (dtype == EPD_F32)
        rc = s.columns == 8    ? launch_rows<norm_backward_kernel<float, 2>>(a, s, grid, stage, st)
             : s.columns == 16 ? launch_rows<norm_backward_kernel<float, 4>>(a, s, grid, stage, st)
                               : launch_rows<norm_backward_kernel<float, 8>>(a, s, grid, stage, st);
    else
        rc = s.columns == 8    ? launch_rows<norm_backward_kernel<__nv_bfloat16, 1>>(a, s, grid, stage, st)
             : s.columns == 16 ? launch_rows<norm_backward_kernel<__nv_bfloat16, 2>>(a, s, grid, stage, st)
                               : launch_rows<norm_backward_kernel<__nv_bfloat16, 4>>(a, s, grid, stage, st);
    if (rc != EPD_OK || !sums || grid == 1) return rc;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((H + 31) / 32), dweight && dbias ? 2 : 1);
    cfg.blockDim = dim3(kReduceThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, norm_reduce_kernel, (const float *)part, grid, a.block_stride, H, dweight, dbias);
    return record_cuda_error();
}
