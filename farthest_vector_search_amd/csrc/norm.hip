// norm.hip -- rows divided by their root mean square, with an addition before
// and 8-bit codes behind, and the gradients.
//
//   h = x + r, rounded to the rows' type (h = x without an addition)
//   rstd = 1 / sqrt(mean_k h_k^2 + eps),  y_k = h_k rstd w_k
//   codes: c_k = the whole number nearest to 127 v_k / max |v|, v = h w in fp32;
//   their scale max |v| rstd / 127.  rstd cancels in the codes, so they follow
//   from h and w alone, and a quotient next to a border is taken again in fp64
//   (exact products, one rounding): the codes do not depend on how sums are cut.
//   backward: with x^ = h rstd and c = mean_k (w dy x^),
//     dx_k = rstd (w_k dy_k - x^_k c) + dh_k,   dw_k = sum over rows dy_k x^_k
// All are bound by memory: a row is read once and held in registers by a wave or
// a workgroup; rows that do not fit are read twice.  Rows of any width are read
// 16 bytes a lane (the part takes such accesses at any address).  Sums are fp32 in a
// fixed order.  A row whose squares leave the range in which fp32 holds them is summed
// again, scaled by a power of two.
#include <type_traits>

#include "vs_internal.h"
#include "vs_types.h"

namespace vs {

namespace {

// 16 bytes of a row at any element boundary.  The lane at `off` of a row of d holds
// elements off .. off + N - 1.  In rows that do not divide (kRagged) the last lane
// holds the row's last N elements, of which those before `off` (the lane's before
// it) read as zeros and are not stored; so do lanes beyond the row.  Loading and
// zeroing are apart, so that loads are issued one behind the other.  Rows of fewer
// than N (kTiny) are one lane's, element by element.
enum Fit { kDivides, kRagged, kTiny };

template <typename T, Fit FIT>
struct Pack {
    static constexpr int N = 16 / (int)sizeof(T);
    typedef T Raw __attribute__((ext_vector_type(N)));
    Raw v;
    static __device__ __forceinline__ int64_t start(int64_t off, int64_t d) {
        return FIT != kRagged || off + N <= d ? off : d - N;
    }
    __device__ __forceinline__ float operator[](int t) const { return widen(v[t]); }
    __device__ __forceinline__ void set(int t, float x) { v[t] = narrow<T>(x); }
    __device__ __forceinline__ void load(const T *row, int64_t off, int64_t d) {
        if constexpr (FIT == kTiny) {
#pragma unroll
            for (int t = 0; t < N; ++t) v[t] = off + t < d ? row[off + t] : T(0.0f);
        } else if (FIT == kRagged || off < d) {
            __builtin_memcpy(&v, row + start(off, d), sizeof(v));
        }
    }
    __device__ __forceinline__ void trim(int64_t off, int64_t d) {
        if constexpr (FIT == kTiny) return;
        if constexpr (FIT == kRagged) {
            const int64_t lost = off - start(off, d);
            if (lost > 0) {
#pragma unroll
                for (int t = 0; t < N; ++t) v[t] = t < lost ? T(0.0f) : v[t];
            }
        } else if (off >= d) {
#pragma unroll
            for (int t = 0; t < N; ++t) v[t] = T(0.0f);
        }
    }
    // the row's element that v[t] holds, -1 where it holds none of its own
    static __device__ __forceinline__ int64_t element(int64_t off, int t, int64_t d) {
        const int64_t at = start(off, d);
        return at + t >= off && at + t < d ? at + t : -1;
    }
    __device__ __forceinline__ void store(T *row, int64_t off, int64_t d) const {
        if (off + N <= d) {
            __builtin_memcpy(row + off, &v, sizeof(v));
        } else if constexpr (FIT != kDivides) {
#pragma unroll
            for (int t = 0; t < N; ++t) {
                const int64_t e = element(off, t, d);
                if (e >= 0) row[e] = v[t];
            }
        }
    }
};

template <typename P>
__device__ __forceinline__ void store_codes(int8_t *row, int64_t off, int64_t d,
                                            const int8_t (&c)[P::N]) {
    if (off + P::N <= d) {
        __builtin_memcpy(row + off, c, P::N);
    } else {
#pragma unroll
        for (int t = 0; t < P::N; ++t) {
            const int64_t e = P::element(off, t, d);
            if (e >= 0) row[e] = c[t];
        }
    }
}

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if one is
    return __builtin_elementwise_maximum(a, b);
}

// (sum, maximum) over the TPR threads of a row, the same in all of them; the
// maximum keeps a NaN
template <int TPR>
__device__ __forceinline__ void row_sum_max(float &s, float &m) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        s += __shfl_xor(s, o);
        m = max_nan(m, __shfl_xor(m, o));
    }
    if constexpr (TPR > 64) {
        __shared__ float part[2][TPR / 64];
        __syncthreads();  // what the last call left has been read
        if ((threadIdx.x & 63) == 0) {
            part[0][threadIdx.x >> 6] = s;
            part[1][threadIdx.x >> 6] = m;
        }
        __syncthreads();
        s = part[0][0];
        m = part[1][0];
#pragma unroll
        for (int w = 1; w < TPR / 64; ++w) {
            s += part[0][w];
            m = max_nan(m, part[1][w]);
        }
    }
}

// The codes of N values of a row whose largest magnitude is top (finite, not 0), inv =
// 127 / top.  Adding 1.5 x 2^23 rounds the quotient and leaves the code in the sum's
// low byte.  The fp32 quotient is within 127 x 4 roundings (3.1e-5) of the exact one; one
// that is this near to a border is taken again in fp64, off by 3e-14 at most.  A quotient
// of two floats, top the larger by 254 at most, that is not on a border is 1e-10 from it
// or more, so 36 binary places tell on, above and below apart.
template <int N>
__device__ __forceinline__ void codes_of(const float (&v)[N], float top, float inv, int8_t (&c)[N]) {
    constexpr float kShift = 0x1.8p23f, kSure = 0.49996f;
    float far = 0.0f;
#pragma unroll
    for (int t = 0; t < N; ++t) {
        const float r = __builtin_fmaf(v[t], inv, kShift);
        c[t] = (int8_t)__builtin_bit_cast(uint32_t, r);
        far = max_nan(far, fabsf(__builtin_fmaf(v[t], inv, kShift - r)));
    }
    if (!(far < kSure)) {
        const double over = 127.0 / (double)top;
#pragma unroll
        for (int t = 0; t < N; ++t) {
            const float q = v[t] * inv;
            if (!(fabsf(q - rintf(q)) < kSure))
                c[t] = (int8_t)(int)rint(rint((double)v[t] * over * 0x1p36) * 0x1p-36);
        }
    }
}

// 1 / sqrt(mean square + eps); 0 where that is not finite (a row of zeros), NaN for a row
// with an infinity or a NaN.  Where ss has left fp32's range, `again(s)` sums (h s)^2, s
// the power of two that takes the row's largest magnitude, top, to 1/2 .. 1.
template <typename F>
__device__ __forceinline__ float rstd_of(float ss, float top, int64_t d, float eps, F again) {
    float rms;
    if (ss >= 0x1p-90f && ss <= 0x1p126f) {
        const float ms = ss / (float)d + eps;
        // an eps near the largest number: the sum of quarters is finite
        rms = ms < __builtin_inff() ? sqrtf(ms) : 2.0f * sqrtf(ss / (float)d * 0.25f + eps * 0.25f);
    } else {
        if (!(top < __builtin_inff())) return __builtin_nanf("");
        int e = top > 0.0f ? __builtin_amdgcn_frexp_expf(top) : 0;
        e = e < -100 ? -100 : e;
        const float a = ldexpf(sqrtf(again(ldexpf(1.0f, -e)) / (float)d), e);
        const float b = sqrtf(eps);
        const float hi = a > b ? a : b, lo = a > b ? b : a;
        rms = hi > 0.0f ? hi * sqrtf(1.0f + (lo / hi) * (lo / hi)) : 0.0f;
    }
    const float r = 1.0f / rms;
    return r < __builtin_inff() || r != r ? r : 0.0f;
}

// threads of a workgroup: four rows of a wave each, or one row
constexpr int block_of(int tpr) { return tpr > 256 ? tpr : 256; }

enum NormOut { kRows, kCodes, kCodesPlain };  // y; codes of y; codes of x itself

template <typename T>
struct NormArgs {
    const T *X, *R, *w;  // R, w may be null
    int64_t n;
    int32_t d;
    float eps;
    T *H;           // with R only
    T *Y;           // kRows
    int8_t *codes;  // the others
    float *scalar;  // rstd (kRows, may be null) or scales
};

// 16,384 rows of 2,048 bf16 with an addition, 268 MB: 44.8 us (6.0 TB/s).  Codes of 8,192
// rows of 8,192, 201 MB: 57 us (3.5 TB/s), bound by a row's loads, sum and stores one
// behind the other in the rows that a CU's registers hold at a time.
//
// VPT vectors a thread, TPR threads a row; VPT = 0: rows of any length, read
// twice.  H may be X or R, Y may be X: every element is read before the thread
// that read it writes it, and a second reading is of h (of x where h is x).
template <typename T, int TPR, int VPT, Fit FIT, NormOut OUT>
__global__ __launch_bounds__(block_of(TPR)) void k_norm_rows(NormArgs<T> a) {
    using P = Pack<T, FIT>;
    constexpr int N = P::N;
    constexpr int kHeld = VPT > 0 ? VPT : 1;
    const int lane = threadIdx.x % TPR;
    const int64_t d = a.d;
    const int turns = VPT > 0 ? VPT : (int)((d + TPR * N - 1) / (TPR * N));
    constexpr int kPer = block_of(TPR) / TPR;  // rows at a time
    const int64_t step = (int64_t)gridDim.x * kPer;
    for (int64_t i = (int64_t)blockIdx.x * kPer + threadIdx.x / TPR; i < a.n; i += step) {
        const T *x = a.X + i * d;
        const bool add_r = a.R != nullptr;
        const T *r = a.R + i * d;
        T *hrow = a.H + i * d;
        P h[kHeld], add[kHeld], w[kHeld];
        float ss = 0.0f, top = 0.0f;
        auto weight = [&](int k, int t) { return a.w ? w[k][t] : 1.0f; };
        auto load_w = [&](int u, int k) {
            if (a.w) w[k].load(a.w, ((int64_t)u * TPR + lane) * N, d);
        };
        auto load = [&](int u, int k) {
            const int64_t off = ((int64_t)u * TPR + lane) * N;
            h[k].load(x, off, d);
            if (add_r) add[k].load(r, off, d);
        };
        auto take = [&](int u, int k) {
            const int64_t off = ((int64_t)u * TPR + lane) * N;
            h[k].trim(off, d);
            if (add_r) add[k].trim(off, d);
            if constexpr (OUT == kCodes)
                if (a.w) w[k].trim(off, d);
#pragma unroll
            for (int t = 0; t < N; ++t) {
                if (add_r) h[k].set(t, h[k][t] + add[k][t]);
                const float f = h[k][t];
                if constexpr (OUT != kCodesPlain) ss = __builtin_fmaf(f, f, ss);
                if constexpr (OUT != kRows)
                    top = max_nan(top, fabsf(OUT == kCodes ? f * weight(k, t) : f));
            }
            if (add_r) h[k].store(hrow, off, d);
        };
        if constexpr (VPT > 0) {
#pragma unroll
            for (int u = 0; u < VPT; ++u) load(u, u);
            if constexpr (OUT != kCodesPlain)
#pragma unroll
                for (int u = 0; u < VPT; ++u) load_w(u, u);
#pragma unroll
            for (int u = 0; u < VPT; ++u) take(u, u);
        } else {
            for (int u = 0; u < turns; ++u) {
                load(u, 0);
                if constexpr (OUT == kCodes) load_w(u, 0);
                take(u, 0);
            }
        }
        row_sum_max<TPR>(ss, top);
        const T *held = add_r ? hrow : x;  // a second reading's rows
        float rstd = 1.0f;
        if constexpr (OUT != kCodesPlain) {
            // the condition, and what the sum needs, are the same in all of a row's threads
            auto sum_scaled = [&](float sc) {
                float s = 0.0f, unused = 0.0f;
#pragma unroll 1
                for (int u = 0; u < turns; ++u) {
                    P p;
                    p.load(held, ((int64_t)u * TPR + lane) * N, d);
                    p.trim(((int64_t)u * TPR + lane) * N, d);
#pragma unroll
                    for (int t = 0; t < N; ++t) {
                        const float f = p[t] * sc;
                        s = __builtin_fmaf(f, f, s);
                    }
                }
                row_sum_max<TPR>(s, unused);
                return s;
            };
            float htop = 0.0f;
            if (!(ss >= 0x1p-90f && ss <= 0x1p126f)) {
                float unused = 0.0f;
#pragma unroll 1
                for (int u = 0; u < turns; ++u) {
                    P p;
                    p.load(held, ((int64_t)u * TPR + lane) * N, d);
                    p.trim(((int64_t)u * TPR + lane) * N, d);
#pragma unroll
                    for (int t = 0; t < N; ++t) htop = max_nan(htop, fabsf(p[t]));
                }
                row_sum_max<TPR>(unused, htop);
            }
            rstd = rstd_of(ss, htop, d, a.eps, sum_scaled);
        }
        const bool coded = top > 0.0f && top < __builtin_inff();
        const float inv = coded ? 127.0f / top : 0.0f;
        auto put = [&](int u, int k) {
            const int64_t off = ((int64_t)u * TPR + lane) * N;
            if constexpr (OUT == kRows) {
                P y;
#pragma unroll
                for (int t = 0; t < N; ++t)
                    y.set(t, h[k][t] * rstd * weight(k, t));
                y.store(a.Y + i * d, off, d);
            } else {
                int8_t c[N] = {};
                float v[N];
#pragma unroll
                for (int t = 0; t < N; ++t) v[t] = OUT == kCodes ? h[k][t] * weight(k, t) : h[k][t];
                if (coded) codes_of(v, top, inv, c);
                store_codes<P>(a.codes + i * d, off, d, c);
            }
        };
        if constexpr (VPT > 0) {
#pragma unroll
            for (int u = 0; u < VPT; ++u) put(u, u);
        } else {
            for (int u = 0; u < turns; ++u) {
                h[0].load(held, ((int64_t)u * TPR + lane) * N, d);
                if constexpr (OUT != kCodesPlain) load_w(u, 0);
                put(u, 0);
            }
        }
        if (lane == 0 && a.scalar) {
            if constexpr (OUT == kRows) {
                a.scalar[i] = rstd;
            } else {
                // a row that holds a NaN or an infinity: NaN, with codes of 0.  top / 127
                // must not become a subnormal number, nor top * rstd an infinity
                const float s = top < 0x1p-100f ? top * rstd / 127.0f : top / 127.0f * rstd;
                a.scalar[i] = coded ? s : top == 0.0f && rstd == rstd ? 0.0f : __builtin_nanf("");
            }
        }
    }
}

template <typename T>
struct NormBwdArgs {
    const T *dY, *H, *w, *dH;  // w, dH may be null
    const float *rstd;
    int64_t n;
    int32_t d;
    T *dX;
    float *part;  // gridDim.x x d partial sums of the weight's gradient, or null
};

// dx needs the row's sum c first, so dy and h stay in registers between the two; the
// weight's gradient is summed there too, over the rows that a thread takes, and stored
// once a workgroup (rows read twice keep it in the workspace).  16,384 rows of 2,048 bf16
// with dH, 268 MB: 43.7 us (6.1 TB/s) and k_norm_join 4.8 us.
template <typename T, int TPR, int VPT, Fit FIT>
__global__ __launch_bounds__(block_of(TPR)) void k_norm_rows_bwd(NormBwdArgs<T> a) {
    using P = Pack<T, FIT>;
    constexpr int N = P::N;
    constexpr int kHeld = VPT > 0 ? VPT : 1;
    constexpr int kPer = block_of(TPR) / TPR;  // rows at a time
    const int lane = threadIdx.x % TPR, mine = threadIdx.x / TPR;
    const int64_t d = a.d;
    const int turns = VPT > 0 ? VPT : (int)((d + TPR * N - 1) / (TPR * N));
    float *part = a.part ? a.part + (int64_t)blockIdx.x * d : nullptr;
    float acc[kHeld][N] = {};
    P w[kHeld], dy[kHeld], h[kHeld], dh[kHeld];
    auto at = [&](int u) { return ((int64_t)u * TPR + lane) * N; };
    auto weight = [&](int k, int t) { return a.w ? w[k][t] : 1.0f; };
    if constexpr (VPT > 0) {
        if (a.w)
#pragma unroll
            for (int u = 0; u < VPT; ++u) w[u].load(a.w, at(u), d);
    }
    const int64_t step = (int64_t)gridDim.x * kPer;
    for (int64_t i0 = (int64_t)blockIdx.x * kPer; i0 < a.n; i0 += step) {
        const int64_t i = i0 + mine;
        if (i >= a.n) break;  // TPR >= 256: uniform over the workgroup
        const T *dyr = a.dY + i * d, *hr = a.H + i * d, *dhr = a.dH + i * d;
        const float rstd = a.rstd[i];
        float dot = 0.0f, unused = 0.0f;
        auto take = [&](int u, int k) {
            dy[k].trim(at(u), d);
            h[k].trim(at(u), d);
            if (a.w) w[k].trim(at(u), d);
#pragma unroll
            for (int t = 0; t < N; ++t)
                dot = __builtin_fmaf(weight(k, t) * dy[k][t], h[k][t] * rstd, dot);
        };
        auto put = [&](int u, int k, float c) {
            P o;
#pragma unroll
            for (int t = 0; t < N; ++t) {
                const float g = dy[k][t], xh = h[k][t] * rstd;
                float v = rstd * (weight(k, t) * g - xh * c);
                if (a.dH) v += dh[k][t];
                o.set(t, v);
            }
            o.store(a.dX + i * d, at(u), d);
        };
        if constexpr (VPT > 0) {
#pragma unroll
            for (int u = 0; u < VPT; ++u) {
                dy[u].load(dyr, at(u), d);
                h[u].load(hr, at(u), d);
            }
            if (a.dH)
#pragma unroll
                for (int u = 0; u < VPT; ++u) dh[u].load(dhr, at(u), d);
#pragma unroll
            for (int u = 0; u < VPT; ++u) take(u, u);
            row_sum_max<TPR>(dot, unused);
            const float c = dot / (float)d;
#pragma unroll
            for (int u = 0; u < VPT; ++u) {
                put(u, u, c);
#pragma unroll
                for (int t = 0; t < N; ++t)
                    acc[u][t] = __builtin_fmaf(dy[u][t], h[u][t] * rstd, acc[u][t]);
            }
        } else {
            for (int u = 0; u < turns; ++u) {
                dy[0].load(dyr, at(u), d);
                h[0].load(hr, at(u), d);
                if (a.w) w[0].load(a.w, at(u), d);
                take(u, 0);
            }
            row_sum_max<TPR>(dot, unused);
            const float c = dot / (float)d;
            for (int u = 0; u < turns; ++u) {
                dy[0].load(dyr, at(u), d);
                h[0].load(hr, at(u), d);
                if (a.w) w[0].load(a.w, at(u), d);
                if (a.dH) dh[0].load(dhr, at(u), d);
                put(u, 0, c);
                // the partial sums of a long row live in the workspace, each
                // element with the thread that owns it
                if (part)
#pragma unroll
                    for (int t = 0; t < N; ++t) {
                        const int64_t e = P::element(at(u), t, d);
                        if (e >= 0) {
                            float *p = part + e;
                            const float before = i0 == (int64_t)blockIdx.x * kPer ? 0.0f : *p;
                            *p = __builtin_fmaf(dy[0][t], h[0][t] * rstd, before);
                        }
                    }
            }
        }
    }
    if constexpr (VPT > 0) {
        if (!part) return;
        if constexpr (kPer > 1) {
            // the waves' sums, added in their order
            __shared__ float sums[kPer][64 * N];
#pragma unroll
            for (int u = 0; u < VPT; ++u) {
                __syncthreads();
#pragma unroll
                for (int t = 0; t < N; ++t) sums[mine][t * 64 + lane] = acc[u][t];
                __syncthreads();
                if (mine == 0)
#pragma unroll
                    for (int t = 0; t < N; ++t) {
                        float s = sums[0][t * 64 + lane];
#pragma unroll
                        for (int v = 1; v < kPer; ++v) s += sums[v][t * 64 + lane];
                        const int64_t e = P::element(at(u), t, d);
                        if (e >= 0) part[e] = s;
                    }
            }
        } else {
#pragma unroll
            for (int u = 0; u < VPT; ++u)
#pragma unroll
                for (int t = 0; t < N; ++t) {
                    const int64_t e = P::element(at(u), t, d);
                    if (e >= 0) part[e] = acc[u][t];
                }
        }
    }
}

// dweight = the partial sums added up: 64 columns a workgroup, its 16 waves take
// the parts in turn and are added in their order.  Few bytes (512 parts of 2,048: 4 MB)
// and few workgroups: bound by the loads' latency, hence eight on their way a wave.
template <typename O>
__global__ __launch_bounds__(1024) void k_norm_join(const float *__restrict__ part, int parts,
                                                    int32_t d, O *__restrict__ dw) {
    __shared__ float sums[16][64];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    float s = 0.0f;
    if (c < d)
#pragma unroll 8
        for (int p = w; p < parts; p += 16) s += part[(int64_t)p * d + c];
    sums[w][lane] = s;
    __syncthreads();
    if (w == 0 && c < d) {
        for (int v = 1; v < 16; ++v) s += sums[v][lane];
        dw[c] = narrow<O>(s);
    }
}

// f(threads a row, vectors a thread, how rows fit the vectors) for n rows of d.
//
// A row is held in registers, by a wave (64) or by a workgroup, in as few threads as keep
// enough rows on their way: a row's latency is what a narrow launch waits for, its
// threads' registers what a wide one does.  us at n rows, bf16 (the chosen side first):
//   d = 1,024    64 threads x 2 against 256 x 1: forward 2,048 rows 5.8, 7.2, 16,384
//                rows 27, 34; 64 rows 3.9, 3.6; backward 512 rows 7.0, 8.5
//   d = 2,048    forward 256 x 1 against 64 x 4: 16,384 rows 48, 50, codes 40, 50; backward
//                64 x 4 against 256 x 1: 16,384 rows 32, 49, 512 rows 9.1, 10.7, 64 rows
//                8.2, 7.1, rows of 1,027 57, 50
//   d = 4,096    256 x 2 against 512 x 1: 8,192 rows 48, 48, codes 33, 44, backward 41, 41
//   d = 8,192    512 x 2 against 256 x 4: 8,192 rows 93, 96, backward 61, 64
//                codes, 8,192 rows: read twice by 256 57, 512 x 2 67; 512 rows 8.1, 7.1
//   d = 16,384   2,048 rows: 512 x 4 53, 1,024 x 2 58, read twice by 256 67; backward 1,024 x
//                2 55, 512 x 4 58, read twice 153; codes: read twice by 256 30, 1,024 x 2 43,
//                64 rows 11.2, 7.1
//   d = 32,768   1,024 x 4 against twice by 1,024: 2,048 rows 109, 114, 64 rows 8.9, 9.7;
//                backward twice, 512 rows 62, 96, 2,048 rows 283, 223 (1,024 x 4 does not
//                fit the registers); codes: twice by 256 against by 1,024, 2,048 rows 71, 74,
//                64 rows 19, 10.6
// A wave holds one row, however narrow, so below 512 columns of 16 bits some of its lanes
// load nothing: 524,288 rows of 128 140 forward, 171 backward (1.9 and 2.4 TB/s), 262,144
// of 64 63 and 82 (1.1 and 1.2 TB/s).
enum Pass { kForward, kToCodes, kBackward };

template <typename T, Pass PASS, typename F>
hipError_t with_row(int64_t n, int32_t d, int n_cu, F f) {
    using std::integral_constant;
    constexpr int N = 16 / (int)sizeof(T);
    const int64_t vecs = ((int64_t)d + N - 1) / N;
    const bool many = n >= (int64_t)n_cu * 4;
    auto go = [&](auto tpr, auto vpt) {
        return d % N ? f(tpr, vpt, integral_constant<Fit, kRagged>())
                     : f(tpr, vpt, integral_constant<Fit, kDivides>());
    };
    integral_constant<int, 0> twice;
    integral_constant<int, 1> v1;
    integral_constant<int, 2> v2;
    integral_constant<int, 4> v4;
    integral_constant<int, 64> t64;
    integral_constant<int, 256> t256;
    integral_constant<int, 512> t512;
    integral_constant<int, 1024> t1024;
    if (d < N) return f(t64, v1, integral_constant<Fit, kTiny>());
    if (vecs <= 64) return go(t64, v1);
    if (vecs <= 128 && (PASS == kBackward || many)) return go(t64, v2);
    if constexpr (PASS == kBackward)
        if (vecs <= 256 && d % N == 0 && n >= (int64_t)n_cu * 2)
            return f(t64, v4, integral_constant<Fit, kDivides>());
    if (vecs <= 256) return go(t256, v1);
    if (vecs <= 512) return go(t256, v2);
    if constexpr (PASS == kToCodes) {
        if (many) return go(t256, twice);
        if (vecs <= 1024) return go(t512, v2);
        if (vecs <= 2048) return go(t1024, v2);
        return go(t1024, twice);
    } else {
        if (vecs <= 1024) return go(t512, v2);
        if (vecs <= 2048) {
            if constexpr (PASS == kForward) return go(t512, v4);
            else return go(t1024, v2);
        }
        if constexpr (PASS == kForward)
            if (vecs <= 4096) return go(t1024, v4);
        return go(t1024, twice);
    }
}

template <typename F>
hipError_t by_type(int dtype, F f) {
    switch (dtype) {
    case kF32: return f(float());
    case kF16: return f(_Float16());
    default: return f(__bf16());
    }
}

template <typename T, NormOut OUT>
hipError_t norm_rows(const NormArgs<T> &a, hipStream_t st, int n_cu) {
    return with_row<T, OUT == kRows ? kForward : kToCodes>(a.n, a.d, n_cu, [&](auto tpr, auto vpt, auto fit) {
        constexpr int TPR = decltype(tpr)::value, VPT = decltype(vpt)::value;
        constexpr int kPer = block_of(TPR) / TPR;
        const int64_t want = (a.n + kPer - 1) / kPer, most = (int64_t)n_cu * 64;
        timing_before(st, OUT == kRows    ? "k_norm_rows"
                          : OUT == kCodes ? "k_norm_rows_q8"
                                          : "k_q8_quantize");
        hipLaunchKernelGGL((k_norm_rows<T, TPR, VPT, decltype(fit)::value, OUT>),
                           dim3((unsigned)(want < most ? want : most)), dim3(block_of(TPR)), 0, st, a);
        timing_after(st);
        return hipGetLastError();
    });
}

// Partial sums of the weight's gradient: one per workgroup of the backward pass.  Fewer
// leave CUs idle, more cost the join.  A workgroup with one vector a thread has half as
// many bytes on their way as one with two, so twice as many of them run (us at 512 and
// 1,024 parts, bf16 unless said: 65,536 x 512 47 and 40, 524,288 x 128 275 and 171, 262,144
// x 64 116 and 80, 16,384 x 2,047 67 and 51, 16,384 x 1,023 fp32 53 and 42, 16,384 x 128
// 12.7 and 13.2; with more vectors: 16,384 x 2,048 40 and 44, 4,096 x 4,096 28 and 32, 65,536
// x 1,024 78 and 84, 16,384 x 1,023 27 and 29).
constexpr int64_t most_parts(int vpt) { return vpt == 1 ? 1024 : 512; }
inline int64_t bwd_groups(int64_t n, int vpt) { return n < most_parts(vpt) ? n : most_parts(vpt); }

}  // namespace

hipError_t launch_norm_rows(const void *X, const void *R, const void *w, int64_t n, int32_t d,
                            int dtype, float eps, void *H, void *Y, float *rstd, hipStream_t st,
                            int n_cu) {
    return by_type(dtype, [&](auto t) {
        using T = decltype(t);
        const NormArgs<T> a{(const T *)X, (const T *)R, (const T *)w, n, d, eps, (T *)H, (T *)Y,
                            nullptr, rstd};
        return norm_rows<T, kRows>(a, st, n_cu);
    });
}

hipError_t launch_norm_rows_q8(const void *X, const void *R, const void *w, int64_t n, int32_t d,
                               int dtype, float eps, void *H, int8_t *codes, float *scales,
                               hipStream_t st, int n_cu) {
    return by_type(dtype, [&](auto t) {
        using T = decltype(t);
        const NormArgs<T> a{(const T *)X, (const T *)R, (const T *)w, n, d, eps, (T *)H, nullptr,
                            codes, scales};
        return norm_rows<T, kCodes>(a, st, n_cu);
    });
}

hipError_t launch_q8_quantize(const void *X, int64_t n, int32_t d, int dtype, int8_t *codes,
                              float *scales, hipStream_t st, int n_cu) {
    return by_type(dtype, [&](auto t) {
        using T = decltype(t);
        const NormArgs<T> a{(const T *)X, nullptr, nullptr, n, d, 0.0f, nullptr, nullptr, codes,
                            scales};
        return norm_rows<T, kCodesPlain>(a, st, n_cu);
    });
}

size_t norm_bwd_workspace(int64_t n, int32_t d) {
    // rows of more than 256 vectors of 16 bits have more than one a thread in every type
    return (size_t)bwd_groups(n, d <= 2048 ? 1 : 2) * (size_t)d * 4;
}

hipError_t launch_norm_rows_bwd(const void *dY, const void *H, const void *w, const void *dH,
                                const float *rstd, int64_t n, int32_t d, int dtype, void *dX,
                                int grad_dtype, void *dw, void *ws, hipStream_t st, int n_cu) {
    int parts = 0;
    const hipError_t e = by_type(dtype, [&](auto t) {
        using T = decltype(t);
        const NormBwdArgs<T> a{(const T *)dY, (const T *)H, (const T *)w, (const T *)dH, rstd, n, d,
                               (T *)dX, dw ? (float *)ws : nullptr};
        if (n == 0) return hipSuccess;
        return with_row<T, kBackward>(n, d, n_cu, [&](auto tpr, auto vpt, auto fit) {
            constexpr int TPR = decltype(tpr)::value, VPT = decltype(vpt)::value;
            constexpr int kPer = block_of(TPR) / TPR;
            const int64_t want = (n + kPer - 1) / kPer, most = bwd_groups(n, VPT);
            parts = (int)(want < most ? want : most);
            timing_before(st, "k_norm_rows_bwd");
            hipLaunchKernelGGL((k_norm_rows_bwd<T, TPR, VPT, decltype(fit)::value>), dim3(parts),
                               dim3(block_of(TPR)), 0, st, a);
            timing_after(st);
            return hipGetLastError();
        });
    });
    if (e != hipSuccess || !dw) return e;
    return by_type(grad_dtype, [&](auto o) {
        using O = decltype(o);
        hipLaunchKernelGGL((k_norm_join<O>), dim3((unsigned)((d + 63) / 64)), dim3(1024), 0, st,
                           (const float *)ws, parts, d, (O *)dw);
        return hipGetLastError();
    });
}

}  // namespace vs
