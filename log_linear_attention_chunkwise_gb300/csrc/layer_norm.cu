// Layer norm over the rows of x [B,H,T,N] with weight and bias [H,N], forward
// and backward.
//
//   y = (x - mean) rstd w + b,   rstd = 1 / sqrt(var + eps)
//   g = dy w,  h = (x - mean) rstd,
//   dx = rstd (g - avg(g) - h avg(g h)),  dw = sum over rows dy h,  db = sum dy
//
// Both directions are bound by memory: every row is read once into registers
// (16-byte pieces where the rows allow it), its sums are formed there in fp32
// (the variance from the centred values, so a large mean costs no digits) and
// it is written once.  TPR threads share a row: 8 to 32 lanes of a warp for
// short rows, a whole CTA for long ones.  Rows are taken ROWS at a time, the
// next ones loading meanwhile, so that enough loads are in flight.  A CTA keeps
// to one (batch, head), whose weights (and, backward, the running column sums
// of dw and db) stay in registers over all of its rows; the CTAs' column sums
// go to the workspace and a second kernel adds them in a fixed order, so
// repeated calls give the same bits.
//
// Measured, whole calls: 16 heads of 32768 rows of 128, bf16, 268 MB, 52 us
// forward (5.2 TB/s; a device copy of the size reaches 6.2); the gradients of 2 x
// 16 heads of 8192 such rows, 201 MB, 39 us; of 8192 rows of 2048, 101 MB, 30 us.
// The figures further down compare variants with one another.
#include "fwd_tc.cuh"
#include "launch.cuh"
#include "layer_norm.cuh"
#include "sm100.cuh"

#include <type_traits>

namespace lla {
namespace {

constexpr int kWarpThreads = 256;  // CTA size of the variants that keep a row within a warp

template <typename T, int VEC> struct Pack;
template <> struct Pack<float, 1> { using type = float; };
template <> struct Pack<float, 4> { using type = float4; };
template <> struct Pack<__nv_bfloat16, 1> { using type = __nv_bfloat16; };
template <> struct Pack<__nv_bfloat16, 8> { using type = uint4; };

template <typename T, int VEC>
__device__ __forceinline__ void unpack(const typename Pack<T, VEC>::type &p, float (&x)[VEC])
{
    const T *e = reinterpret_cast<const T *>(&p);
#pragma unroll
    for (int i = 0; i < VEC; i++) x[i] = to_f32<T>(e[i]);
}

template <typename T, int VEC>
__device__ __forceinline__ typename Pack<T, VEC>::type pack(const float (&x)[VEC])
{
    typename Pack<T, VEC>::type p;
    T *e = reinterpret_cast<T *>(&p);
#pragma unroll
    for (int i = 0; i < VEC; i++) e[i] = from_f32<T>(x[i]);
    return p;
}

// VEC fp32 values of a [N] vector at column c, or `other` without a vector.
template <int VEC>
__device__ __forceinline__ void load_param(const float *p, int c, float other, float (&x)[VEC])
{
    if (p == nullptr) {
#pragma unroll
        for (int i = 0; i < VEC; i++) x[i] = other;
    } else if constexpr (VEC % 4 == 0) {
#pragma unroll
        for (int i = 0; i < VEC; i += 4) *reinterpret_cast<float4 *>(&x[i]) = *reinterpret_cast<const float4 *>(p + c + i);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; i++) x[i] = p[c + i];
    }
}

// Sums of M values over the TPR threads that share rows, in every thread.
// Within a warp by shuffles; over a CTA through `red` (M per warp), one barrier:
// the caller alternates between two such buffers, so that the barrier of one
// sum also says that the last one has been read.
template <int TPR, int M>
__device__ __forceinline__ void row_sum(float (&v)[M], float *red)
{
#pragma unroll
    for (int off = (TPR < 32 ? TPR : 32) / 2; off > 0; off >>= 1)
#pragma unroll
        for (int i = 0; i < M; i++) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
    if constexpr (TPR > 32) {
        constexpr int kWarps = TPR / 32;
        const int w = threadIdx.x >> 5;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < M; i++) red[i * kWarps + w] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < M; i++) {
            float t = 0.f;
            if constexpr (kWarps % 4 == 0) {
#pragma unroll
                for (int j = 0; j < kWarps; j += 4) {
                    const float4 q = *reinterpret_cast<const float4 *>(red + i * kWarps + j);
                    t += (q.x + q.y) + (q.z + q.w);
                }
            } else {
#pragma unroll
                for (int j = 0; j < kWarps; j++) t += red[i * kWarps + j];
            }
            v[i] = t;
        }
    }
}

// A ring of kStages turns' rows in shared memory, filled by bulk copies (rows of
// a chunk are contiguous, so a turn is one copy an input): what keeps enough
// bytes in flight without holding them in registers.  Used where rows are whole
// 16-byte pieces and a turn of all inputs fits kRingBytes at least twice.
constexpr int kRingBytes = 40 * 1024;
constexpr uint32_t kCopyWait = 1u << 18;  // bounded waits (about half a second: 1.7 us a poll)
constexpr uint32_t kGivenUp = 16;         // of a CTA one of whose waits ran out,
constexpr uint32_t kDrained = 15;         // and whose filling thread has seen to what was in flight

template <int INPUTS, int TURN_BYTES>
struct Ring {
    static constexpr int kFit = kRingBytes / (INPUTS * TURN_BYTES);
    static constexpr int kStages = kFit > 4 ? 4 : kFit;
    uint8_t data[kStages][INPUTS][TURN_BYTES];
    uint64_t bar[kStages];
    volatile uint32_t limit;  // polls of a wait

    __device__ __forceinline__ void init()
    {
        if (threadIdx.x == 0) {
            limit = kCopyWait;
            for (int i = 0; i < kStages; i++) sm100::mbar_init(&bar[i], 1);
            sm100::fence_mbar_init();
        }
        __syncthreads();
    }
    // one thread: turn t's `bytes` of every input.  Not once a wait has run out: the barrier may still count the
    // place's last copy.
    __device__ __forceinline__ void fill(int t, const void *const (&src)[INPUTS], uint32_t bytes)
    {
        if (limit != kCopyWait) return;
        uint64_t *b = &bar[t % kStages];
        sm100::mbar_arrive_expect_tx(b, INPUTS * bytes);
        for (int k = 0; k < INPUTS; k++) sm100::bulk_load(data[t % kStages][k], src[k], bytes, b);
    }
    __device__ __forceinline__ void wait(int t, int32_t *err)
    {
        if (!sm100::mbar_try_wait(&bar[t % kStages], (t / kStages) & 1)) wait_on(t, err);
    }
    // out of line, for the registers of the loops that wait
    __device__ __noinline__ void wait_on(int t, int32_t *err)
    {
        if (sm100::mbar_wait(&bar[t % kStages], (t / kStages) & 1, limit)) return;
        if (err != nullptr) atomicCAS(err, 0, LLA_DEVERR_COPY_TIMEOUT);
        // Later waits are short.  The thread that fills waits here, once, for all that may be in flight (turns not
        // asked for take their limit), so that none is when the CTA ends.
        if (threadIdx.x == 0 && limit != kDrained) {
            limit = kDrained;
            for (int i = 0; i < kStages; i++, t++) sm100::mbar_wait(&bar[t % kStages], (t / kStages) & 1, kCopyWait);
        } else if (limit == kCopyWait) {
            limit = kGivenUp;
        }
    }
};

struct NormParams {
    const void *x, *dy;
    const float *weight, *bias;
    const int32_t *lens;
    void *y;
    float *mean, *rstd;
    float *part;      // backward: [H][CTAs of a head][2][N]
    long long rows_per_cta;
    int H, T, N, chunks;  // chunks: CTAs of one (batch, head)
    float eps;
    int32_t *err;
    int withhold;         // test hook: the ring's first copy is not issued
};

// Rows of (b, h) that count: lens[b], T without lens; a length out of range is
// reported and the sequence skipped.
__device__ __forceinline__ int rows_of(const int32_t *lens, int b, int T, int32_t *err)
{
    if (lens == nullptr) return T;
    const int n = lens[b];
    if (n >= 0 && n <= T) return n;
    if (err != nullptr && threadIdx.x == 0) atomicCAS(err, 0, LLA_DEVERR_BAD_LENGTH);
    return 0;
}

template <typename T, int VEC, int TPR, int ITEMS, int ROWS, int THREADS>
__global__ void __launch_bounds__(THREADS)
layer_norm_fwd_kernel(const __grid_constant__ NormParams p)
{
    using P = typename Pack<T, VEC>::type;
    constexpr int kGroups = THREADS / TPR, kTurn = kGroups * ROWS;
    __shared__ __align__(16) float red[2][TPR > 32 ? ROWS * (TPR / 32) : 1];
    const long long bh = blockIdx.x / p.chunks;
    const int chunk = (int)(blockIdx.x % p.chunks);
    const int h = (int)(bh % p.H), b = (int)(bh / p.H);
    const int n = rows_of(p.lens, b, p.T, p.err);
    const long long lo = chunk * p.rows_per_cta;
    const long long hi = min((long long)n, lo + p.rows_per_cta);
    const int lane = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    const int N = p.N, np = N / VEC;
    const T *x = (const T *)p.x + bh * p.T * N;
    T *y = (T *)p.y + bh * p.T * N;
    const float *wp = p.weight ? p.weight + (long long)h * N : nullptr;
    const float *bp = p.bias ? p.bias + (long long)h * N : nullptr;
    float w[ITEMS][VEC], bb[ITEMS][VEC];
#pragma unroll
    for (int i = 0; i < ITEMS; i++) {
        const int c = lane + i * TPR;
        if (c < np) {
            load_param<VEC>(wp, c * VEC, 1.f, w[i]);
            load_param<VEC>(bp, c * VEC, 0.f, bb[i]);
        }
    }
    const float inv = 1.f / (float)N;
    constexpr int kTurnBytes = THREADS * ROWS * ITEMS * VEC * (int)sizeof(T);
    constexpr bool kBulk = VEC > 1 && 2 * kTurnBytes <= kRingBytes;
    __shared__ __align__(128) std::conditional_t<kBulk, Ring<1, kTurnBytes>, int> ring;
    [[maybe_unused]] auto fill = [&](int t) {
        const long long r = lo + (long long)t * kTurn;
        const void *const src[1] = {x + r * N};
        if constexpr (kBulk)
            if (r < hi && (t > 0 || !p.withhold)) ring.fill(t, src, (uint32_t)(min((long long)kTurn, hi - r) * N * sizeof(T)));
    };
    auto load = [&](long long r0, int t, P (&raw)[ROWS][ITEMS]) {
#pragma unroll
        for (int q = 0; q < ROWS; q++)
#pragma unroll
            for (int i = 0; i < ITEMS; i++) {
                const int k = q * kGroups + grp;
                const int c = lane + i * TPR;
                raw[q][i] = P{};
                if (r0 + k >= hi || c >= np) continue;
                if constexpr (kBulk)
                    raw[q][i] = reinterpret_cast<const P *>(ring.data[t % ring.kStages][0])[k * np + c];
                else
                    raw[q][i] = reinterpret_cast<const P *>(x + (r0 + k) * N)[c];
            }
    };
    P raw[ROWS][ITEMS];
    if constexpr (kBulk) {
        ring.init();
        if (threadIdx.x == 0)
            for (int t = 0; t < ring.kStages; t++) fill(t);
    } else {
        load(lo, 0, raw);
    }
    // every thread of the CTA takes the same number of turns (row_sum synchronises)
    int t = 0;
    for (long long r0 = lo; r0 < hi; r0 += kTurn, t++) {
        [[maybe_unused]] P next[ROWS][ITEMS];
        if constexpr (kBulk) {
            ring.wait(t, p.err);
            load(r0, t, raw);
        } else {
            load(r0 + kTurn, 0, next);  // on their way while this turn's rows are worked on
        }
        float sum[ROWS], sq[ROWS];
#pragma unroll
        for (int q = 0; q < ROWS; q++) {
            sum[q] = 0.f;
#pragma unroll
            for (int i = 0; i < ITEMS; i++) {
                float v[VEC];
                unpack<T, VEC>(raw[q][i], v);
#pragma unroll
                for (int e = 0; e < VEC; e++) sum[q] += v[e];
            }
        }
        row_sum<TPR, ROWS>(sum, red[0]);
        if constexpr (kBulk) {
            // the stage has been read: every thread has the values themselves, not only reads under way
            if constexpr (TPR <= 32) __syncthreads();
            if (threadIdx.x == 0) fill(t + ring.kStages);
        }
#pragma unroll
        for (int q = 0; q < ROWS; q++) {
            sum[q] *= inv;
            sq[q] = 0.f;
#pragma unroll
            for (int i = 0; i < ITEMS; i++)
                if (lane + i * TPR < np) {
                    float v[VEC];
                    unpack<T, VEC>(raw[q][i], v);
#pragma unroll
                    for (int e = 0; e < VEC; e++) {
                        const float d = v[e] - sum[q];
                        sq[q] = fmaf(d, d, sq[q]);
                    }
                }
        }
        row_sum<TPR, ROWS>(sq, red[1]);
#pragma unroll
        for (int q = 0; q < ROWS; q++) {
            const long long r = r0 + q * kGroups + grp;
            if (r >= hi) continue;
            const float rs = rsqrtf(fmaf(sq[q], inv, p.eps));
#pragma unroll
            for (int i = 0; i < ITEMS; i++) {
                const int c = lane + i * TPR;
                if (c >= np) continue;
                float v[VEC];
                unpack<T, VEC>(raw[q][i], v);
#pragma unroll
                for (int e = 0; e < VEC; e++) v[e] = fmaf((v[e] - sum[q]) * rs, w[i][e], bb[i][e]);
                reinterpret_cast<P *>(y + r * N)[c] = pack<T, VEC>(v);
            }
            if (lane == 0) {
                if (p.mean) p.mean[bh * p.T + r] = sum[q];
                if (p.rstd) p.rstd[bh * p.T + r] = rs;
            }
        }
        if constexpr (!kBulk)
#pragma unroll
            for (int q = 0; q < ROWS; q++)
#pragma unroll
                for (int i = 0; i < ITEMS; i++) raw[q][i] = next[q][i];
    }
}

// CTAs of the backward an SM holds: the fewest that keep enough bytes in flight,
// since every CTA leaves a row of column sums for each gradient.  Three of 256
// threads where a row stays within a warp and a thread has 16 bytes of it (2 x
// 16 heads of 8192 rows of 128, bf16: 40 us with two, 37 with three, 113 with
// four, whose registers no longer hold a turn; with 32 bytes three no longer
// hold one either: 131072 rows of 256, fp32, 154 us with three, 73 with two),
// else 512 threads (8192 rows of 2048: 28 us so, 33 with 768, 60 with 1024).
template <typename T, int TPR, int VEC, int ITEMS, int THREADS>
constexpr int kBwdCtas =
    TPR <= 32 && (VEC > 1 ? VEC * ITEMS * sizeof(T) <= 16 : ITEMS <= 4) ? 3 : (THREADS < 512 ? 512 / THREADS : 1);

template <typename T, int VEC, int TPR, int ITEMS, int ROWS, int THREADS>
__global__ void __launch_bounds__(THREADS, kBwdCtas<T, TPR, VEC, ITEMS, THREADS>)
layer_norm_bwd_kernel(const __grid_constant__ NormParams p)
{
    using P = typename Pack<T, VEC>::type;
    constexpr int kGroups = THREADS / TPR, kTurn = kGroups * ROWS;
    // row groups' column sums, added when the rows are done
    __shared__ float col[kGroups > 1 ? kGroups : 1][TPR > 32 ? 1 : TPR * VEC];
    __shared__ __align__(16) float red[2][TPR > 32 ? 2 * ROWS * (TPR / 32) : 1];
    const long long bh = blockIdx.x / p.chunks;
    const int chunk = (int)(blockIdx.x % p.chunks);
    const int h = (int)(bh % p.H), b = (int)(bh / p.H);
    const int n = rows_of(p.lens, b, p.T, p.err);
    const unsigned lo = (unsigned)(chunk * p.rows_per_cta);  // rows fit 32 bits, a turn beyond T too
    const unsigned hi = (unsigned)min((long long)n, chunk * p.rows_per_cta + p.rows_per_cta);
    const int lane = threadIdx.x % TPR, grp = threadIdx.x / TPR;
    const int N = p.N, np = N / VEC;
    sm100::grid_launch_dependents();
    const T *x = (const T *)p.x + bh * p.T * N;
    const T *dy = (const T *)p.dy + bh * p.T * N;
    T *dx = (T *)p.y + bh * p.T * N;
    const float *mean = p.mean + bh * p.T, *rstd = p.rstd + bh * p.T;
    const float *wp = p.weight ? p.weight + (long long)h * N : nullptr;
    float w[ITEMS][VEC], dw[ITEMS][VEC], db[ITEMS][VEC];
#pragma unroll
    for (int i = 0; i < ITEMS; i++) {
#pragma unroll
        for (int e = 0; e < VEC; e++) w[i][e] = dw[i][e] = db[i][e] = 0.f;
        const int c = lane + i * TPR;
        if (c < np) load_param<VEC>(wp, c * VEC, 1.f, w[i]);
    }
    const float inv = 1.f / (float)N;
    constexpr int kTurnBytes = THREADS * ROWS * ITEMS * VEC * (int)sizeof(T);
    constexpr bool kBulk = VEC > 1 && 4 * kTurnBytes <= kRingBytes;
    __shared__ __align__(128) std::conditional_t<kBulk, Ring<2, kTurnBytes>, int> ring;
    [[maybe_unused]] auto fill = [&](int t) {
        const unsigned r = lo + (unsigned)t * kTurn;
        const void *const src[2] = {x + (long long)r * N, dy + (long long)r * N};
        if constexpr (kBulk)
            if (r < hi && (t > 0 || !p.withhold)) ring.fill(t, src, (uint32_t)(min((unsigned)kTurn, hi - r) * N * (unsigned)sizeof(T)));
    };
    struct Rows {
        P x[ROWS][ITEMS], d[ROWS][ITEMS];
        float mu[ROWS], rs[ROWS];
    };
    auto load_stats = [&](unsigned r0, Rows &t) {
#pragma unroll
        for (int q = 0; q < ROWS; q++) {
            const unsigned r = r0 + q * kGroups + grp;
            t.mu[q] = r < hi ? mean[r] : 0.f;
            t.rs[q] = r < hi ? rstd[r] : 0.f;
        }
    };
    auto load_rows = [&](unsigned r0, int n, Rows &t) {
#pragma unroll
        for (int q = 0; q < ROWS; q++)
#pragma unroll
            for (int i = 0; i < ITEMS; i++) {
                const int k = q * kGroups + grp;
                const int c = lane + i * TPR;
                t.x[q][i] = t.d[q][i] = P{};
                if (r0 + k >= hi || c >= np) continue;
                if constexpr (kBulk) {
                    t.x[q][i] = reinterpret_cast<const P *>(ring.data[n % ring.kStages][0])[k * np + c];
                    t.d[q][i] = reinterpret_cast<const P *>(ring.data[n % ring.kStages][1])[k * np + c];
                } else {
                    t.x[q][i] = reinterpret_cast<const P *>(x + (long long)(r0 + k) * N)[c];
                    t.d[q][i] = reinterpret_cast<const P *>(dy + (long long)(r0 + k) * N)[c];
                }
            }
    };
    Rows t;
    if constexpr (kBulk) {
        ring.init();
        if (threadIdx.x == 0)
            for (int n = 0; n < ring.kStages; n++) fill(n);
    } else {
        load_rows(lo, 0, t);
    }
    load_stats(lo, t);
    int turn = 0, n_turn = 0;
    for (unsigned r0 = lo; r0 < hi; r0 += kTurn, turn ^= 1, n_turn++) {
        Rows next;  // on their way while these rows are worked on
        load_stats(r0 + kTurn, next);
        if constexpr (kBulk) {
            ring.wait(n_turn, p.err);
            load_rows(r0, n_turn, t);
        } else {
            load_rows(r0 + kTurn, 0, next);
        }
        float s[2 * ROWS];
        // a row beyond hi has rstd 0 and dy 0, a column beyond N has dy 0 and w 0:
        // neither adds to any sum
#pragma unroll
        for (int q = 0; q < ROWS; q++) {
            float s1 = 0.f, s2 = 0.f;
#pragma unroll
            for (int i = 0; i < ITEMS; i++) {
                float xv[VEC], dv[VEC];
                unpack<T, VEC>(t.x[q][i], xv);
                unpack<T, VEC>(t.d[q][i], dv);
#pragma unroll
                for (int e = 0; e < VEC; e++) {
                    const float hh = (xv[e] - t.mu[q]) * t.rs[q], g = __fmul_rn(dv[e], w[i][e]);
                    s1 += g;
                    s2 = fmaf(g, hh, s2);
                    dw[i][e] = fmaf(dv[e], hh, dw[i][e]);
                    db[i][e] += dv[e];
                }
            }
            s[2 * q] = s1;
            s[2 * q + 1] = s2;
        }
        row_sum<TPR, 2 * ROWS>(s, red[turn]);
        if constexpr (kBulk) {
            // the stage has been read: every thread has the values themselves, not only reads under way
            if constexpr (TPR <= 32) __syncthreads();
            if (threadIdx.x == 0) fill(n_turn + ring.kStages);
        }
#pragma unroll
        for (int q = 0; q < ROWS; q++) {
            const unsigned r = r0 + q * kGroups + grp;
            if (r >= hi) continue;
            const float a = s[2 * q] * inv, c2 = s[2 * q + 1] * inv;
#pragma unroll
            for (int i = 0; i < ITEMS; i++) {
                const int c = lane + i * TPR;
                if (c >= np) continue;
                float xv[VEC], dv[VEC], o[VEC];
                unpack<T, VEC>(t.x[q][i], xv);
                unpack<T, VEC>(t.d[q][i], dv);
#pragma unroll
                for (int e = 0; e < VEC; e++) {
                    const float hh = (xv[e] - t.mu[q]) * t.rs[q];
                    // g rounded as in its sum: what cancels exactly (a row of one column) leaves nothing
                    o[e] = t.rs[q] * ((__fmul_rn(dv[e], w[i][e]) - a) - hh * c2);
                }
                reinterpret_cast<P *>(dx + (long long)r * N)[c] = pack<T, VEC>(o);
            }
        }
        if constexpr (kBulk) {
#pragma unroll
            for (int q = 0; q < ROWS; q++) {
                t.mu[q] = next.mu[q];
                t.rs[q] = next.rs[q];
            }
        } else {
            t = next;
        }
    }
    if (p.part == nullptr) return;
    // this CTA's column sums: [h][b * chunks + chunk][dw | db][N]
    const long long nb = (long long)(gridDim.x / p.H);
    float *part = p.part + ((long long)h * nb + (long long)b * p.chunks + chunk) * 2 * N;
    if constexpr (TPR > 32) {  // one row group: the thread's own columns
#pragma unroll
        for (int i = 0; i < ITEMS; i++) {
            const int c = (lane + i * TPR) * VEC;
            if (c >= N) continue;
#pragma unroll
            for (int e = 0; e < VEC; e++) {
                part[c + e] = dw[i][e];
                part[N + c + e] = db[i][e];
            }
        }
    } else {
        for (int which = 0; which < 2; which++)
#pragma unroll
            for (int i = 0; i < ITEMS; i++) {
                __syncthreads();
#pragma unroll
                for (int e = 0; e < VEC; e++) col[grp][lane * VEC + e] = which ? db[i][e] : dw[i][e];
                __syncthreads();
                for (int j = threadIdx.x; j < TPR * VEC; j += THREADS) {
                    const int c = i * TPR * VEC + j;
                    if (c >= N) continue;
                    float t = 0.f;
                    for (int g = 0; g < kGroups; g++) t += col[g][j];
                    part[which * N + c] = t;
                }
            }
    }
}

// dweight, dbias [H][N] from nb parts [H][nb][2][N]: 32 columns a CTA, 32
// threads down each, every thread adding every 32nd part in order and the 32
// sums in order.  `part` is no __restrict__ pointer: loads taken for constant
// could be moved ahead of the wait.
constexpr int kDown = 32;

__global__ void __launch_bounds__(32 * kDown)
layer_norm_param_kernel(const float *part, float *dweight, float *dbias, int nb, int N, int cols)
{
    __shared__ float red[kDown][33];
    const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
    const int h = blockIdx.x / cols, c = (blockIdx.x % cols) * 32 + cx;
    const int which = blockIdx.y;
    sm100::grid_dependency_wait();  // the parts are the kernel's before this one
    float t = 0.f;
    if (c < N) {
        const float *p = part + ((long long)h * nb * 2 + which) * N + c;
#pragma unroll 8
        for (int j = ry; j < nb; j += kDown) t += p[(long long)j * 2 * N];
    }
    red[ry][cx] = t;
    __syncthreads();
    float *dst = which ? dbias : dweight;
    if (ry == 0 && c < N && dst != nullptr) {
#pragma unroll
        for (int j = 1; j < kDown; j++) t += red[j][cx];
        dst[(long long)h * N + c] = t;
    }
}

// One compiled variant: a row of up to TPR * ITEMS * VEC values.
struct Variant {
    int cap, threads, fwd_turn, bwd_turn;  // rows a CTA takes at a time
    int bwd_ctas;                          // per SM
    void (*fwd)(NormParams);
    void (*bwd)(NormParams);
};

template <typename T, int VEC, int TPR, int ITEMS>
constexpr Variant variant()
{
    constexpr int kThreads = TPR > 32 ? TPR : kWarpThreads;
    constexpr int kHeld = ITEMS * VEC;  // values of a row a thread holds
    constexpr int kRows = TPR > 32 ? (kHeld <= 8 && TPR < 1024 ? 2 : 1) : (kHeld <= 8 ? 4 : (kHeld <= 16 ? 2 : 1));
    constexpr int kRowsB = kHeld <= 8 && TPR < 1024 ? 2 : 1;
    return {TPR * ITEMS * VEC, kThreads, kThreads / TPR * kRows, kThreads / TPR * kRowsB, kBwdCtas<T, TPR, VEC, ITEMS, kThreads>,
            layer_norm_fwd_kernel<T, VEC, TPR, ITEMS, kRows, kThreads>,
            layer_norm_bwd_kernel<T, VEC, TPR, ITEMS, kRowsB, kThreads>};
}

template <typename T> struct Variants;
template <> struct Variants<__nv_bfloat16> {
    static constexpr int kVec = 8;
    static const Variant *wide()
    {
        using T = __nv_bfloat16;
        static const Variant v[] = {variant<T, 8, 8, 1>(),   variant<T, 8, 16, 1>(),  variant<T, 8, 32, 1>(),
                                    variant<T, 8, 32, 2>(),  variant<T, 8, 128, 1>(), variant<T, 8, 256, 1>(),
                                    variant<T, 8, 512, 1>(), variant<T, 8, 512, 2>(), variant<T, 8, 1024, 2>()};
        return v;
    }
};
template <> struct Variants<float> {
    static constexpr int kVec = 4;
    static const Variant *wide()
    {
        using T = float;
        static const Variant v[] = {variant<T, 4, 8, 1>(),   variant<T, 4, 16, 1>(),  variant<T, 4, 32, 1>(),
                                    variant<T, 4, 32, 2>(),  variant<T, 4, 32, 4>(),  variant<T, 4, 256, 1>(),
                                    variant<T, 4, 512, 1>(), variant<T, 4, 512, 2>(), variant<T, 4, 512, 4>(),
                                    variant<T, 4, 1024, 4>()};
        return v;
    }
};

// The narrowest variant that holds a row.  Rows whose length is no multiple of
// a 16-byte piece go value by value (VEC = 1).
// Above 8192 columns a thread keeps 16 values in 64 registers and spills a part
// of them; odd widths up to there have a variant of 8 and a row a turn (4000 rows
// of 5001, bf16: 92 and 333 us forward and backward in the wide one, 48 and 96 in
// this).
template <typename T>
const Variant &pick(int N)
{
    static const Variant narrow[] = {variant<T, 1, 8, 1>(),   variant<T, 1, 32, 1>(),  variant<T, 1, 32, 4>(),
                                     variant<T, 1, 32, 8>(),  variant<T, 1, 128, 8>(), variant<T, 1, 512, 8>(),
                                     variant<T, 1, 1024, 8>(), variant<T, 1, 1024, 16>()};
    const Variant *v = N % Variants<T>::kVec == 0 ? Variants<T>::wide() : narrow;
    while (v->cap < N) v++;
    return *v;
}

// CTAs of one (batch, head) and the rows of each: at most `per_sm` CTAs per SM
// over the grid and at least one turn each.  Backward that is what an SM holds (a
// CTA more would wait for a whole one to end and leave another row of sums).
void split_rows(int turn, int B, int H, int T, int per_sm, long long *rows_per_cta, int *chunks)
{
    const long long bh = (long long)B * H;
    const long long turns = ((long long)T + turn - 1) / turn;
    long long c = (long long)sm_count() * per_sm / bh;
    c = c < 1 ? 1 : (c > turns ? turns : c);
    *rows_per_cta = (turns + c - 1) / c * turn;
    *chunks = (int)(((long long)T + *rows_per_cta - 1) / *rows_per_cta);
}

// Forward, threads of a full SM: more than the registers hold (768), on purpose: the rest of the grid fills the
// places of CTAs that have ended (65536 rows of 2048: 95 us so, 100 with 768 threads' CTAs).
int fwd_ctas(const Variant &v) { return 2048 / v.threads; }

NormParams params(const LayerNormArgs &A, const Variant &v, bool bwd)
{
    NormParams p{};
    p.x = A.x; p.dy = A.dy; p.weight = A.weight; p.bias = A.bias; p.lens = A.lens; p.y = A.y;
    p.mean = A.mean; p.rstd = A.rstd; p.H = A.H; p.T = A.T; p.N = A.N; p.eps = A.eps; p.err = A.device_error;
    p.withhold = withhold_first_product() ? 1 : 0;
    split_rows(bwd ? v.bwd_turn : v.fwd_turn, A.B, A.H, A.T, bwd ? v.bwd_ctas : fwd_ctas(v),
               &p.rows_per_cta, &p.chunks);
    return p;
}

const Variant &pick(int N, lla_dtype dt) { return dt == LLA_BF16 ? pick<__nv_bfloat16>(N) : pick<float>(N); }

}  // namespace

cudaError_t layer_norm_fwd(const LayerNormArgs &A)
{
    const Variant &v = pick(A.N, A.dt);
    const NormParams p = params(A, v, false);
    const unsigned grid = (unsigned)((long long)A.B * A.H * p.chunks);
    v.fwd<<<grid, v.threads, 0, (cudaStream_t)A.stream>>>(p);
    return cudaPeekAtLastError();
}

size_t layer_norm_bwd_workspace_bytes(int B, int H, int T, int N, lla_dtype dt)
{
    const Variant &v = pick(N, dt);
    long long rows;
    int chunks;
    split_rows(v.bwd_turn, B, H, T, v.bwd_ctas, &rows, &chunks);
    return align_up((size_t)B * H * chunks * 2 * N * sizeof(float), 256);
}

cudaError_t layer_norm_bwd(const LayerNormArgs &A)
{
    const Variant &v = pick(A.N, A.dt);
    NormParams p = params(A, v, true);
    const bool sums = A.dweight != nullptr || A.dbias != nullptr;
    p.part = sums ? (float *)A.workspace : nullptr;
    const unsigned grid = (unsigned)((long long)A.B * A.H * p.chunks);
    v.bwd<<<grid, v.threads, 0, (cudaStream_t)A.stream>>>(p);
    cudaError_t e = cudaPeekAtLastError();
    if (e != cudaSuccess || !sums) return e;
    const int cols = (A.N + 31) / 32;
    return launch_kernel(layer_norm_param_kernel, dim3((unsigned)(A.H * cols), 2), 32 * kDown, 0, A.stream, true,
                         (const float *)p.part, A.dweight, A.dbias, A.B * p.chunks, A.N, cols);
}

}  // namespace lla
