// Linear attention with one decay per head on the 5th-generation tensor cores
// (tcgen05, tensor memory, TMA): bf16, dk and dv up to D = 64 or 128.
//
// Narrower inputs are padded to D on the chip: the loads fill the columns that
// are not there with zeros and the stores leave them out, so that no byte more
// is moved, and products of zeros are what the memory's time hides anyway.
//
// A CTA walks one segment of one (job, batch, head) in tiles of 128 tokens
// with the state U (D x D, fp32) in tensor memory.  Per tile of n tokens, with
// the walk's inputs x, y, z (linattn.cuh) and w, u the powers of the decay:
//   S   = X Y^T                              P_ij = a^|i-j| S_ij, masked, bf16
//   O   = X bf16(U), rows times w_i in place, then O += P Z (P is the A operand in
//         tensor memory)
//   U   = a^n U + (diag(u) Y)^T Z            diag(u) Y in bf16 parts
// so each input is read and each output written once.  P and the read-out's
// copy of U are rounded once to bf16 (as the output is).  y and z are exact in
// bf16; u y goes in two parts (16 bits), far below that rounding.  A state that
// is handed out comes from the state pass below, in fp32 accuracy.
//
// Bound, where every SM has a walk, by memory: 8 D bytes a token and head (4
// rows of bf16); elsewhere by the chain from one tile's state to the next,
// 3.0 us at D = 128: U out of tensor memory into its operand, the read-out,
// its scaling, P Z.  So what matters is what stands between the products, and
// two groups of warps work side by side, two threads per row each: eight warps
// turn S into P and drain the output, eight hand U to the read-out and split
// u y.  Four single threads issue: the loads of x and y (the next tile's rows
// are brought to L2 meanwhile), the scores' products, the outputs' way out
// with the loads of z into the places they leave, and the state's products; so
// neither chain of products waits for the other's.  Shared memory holds the
// state operand, both parts, x, y and two stages of z, 32 KB each at D = 128.
//
// Measured: 16 heads of 32768 tokens, D = 128, in 9 segments each 102 us for
// 537 MB (5.3 TB/s; the state pass before it 61 us for 268 MB; the call 169);
// 128 whole walks of 2500 tokens 72 us; the gradients' 96 whole walks of 8192
// tokens 196 us.
// The simple kernel on the CUDA cores took 2322 us for the first, state and all.
#include "launch.cuh"
#include "linattn.cuh"
#include "sm100.cuh"
#include "tma_host.cuh"

namespace lla {
namespace {

using namespace sm100;

constexpr int kTile = kLinTile;
constexpr int kStages = 2;
constexpr uint32_t kBlk = kTile * 128;      // a 64-column block of a 128-row bf16 tile
constexpr uint32_t kWait = 1u << 18;        // bounded waits (about half a second: 1.7 us a poll)
constexpr uint32_t kIssuerSpin = 1u << 22;  // the scores' issuer's polls
constexpr uint32_t kGivenUp = 16;           // of a thread one of whose waits ran out
constexpr int kRowWarps = 8, kStateWarps = 8;
constexpr int kWalkThreads = (kRowWarps + kStateWarps + 4) * 32;
constexpr int kLoadThread = (kRowWarps + kStateWarps) * 32, kStoreThread = kLoadThread + 2 * 32;  // roles 0 and 2
constexpr int kSumWarps = 16;  // four threads per token row
constexpr int kSumThreads = (kSumWarps + 2) * 32;

struct WalkMaps {
    CUtensorMap x[kLinMaxJobs], y[kLinMaxJobs], z[kLinMaxJobs], out[kLinMaxJobs];
};

template <int D>
struct __align__(1024) WalkSmem {
    // first the three whose D = 64 products read past their end
    uint8_t u[kTile * D * 2];   // U in bf16 [D][D]
    uint8_t hi[kTile * D * 2];  // the high and the middle part of u y
    uint8_t mid[kTile * D * 2];
    uint8_t x[kTile * D * 2];
    uint8_t y[kTile * D * 2];
    uint8_t z[kStages][kTile * D * 2];  // Z; then the output on its way out
    float pw[kTile + 4];  // a^n
    float cf[32];         // a full 32-column block's factors: a^(31-c) forward, a^c backward
    float diag[64];       // a diagonal block's by distance + 32: 0 on the masked side, else a^distance
    uint64_t bar_x, bar_y, bar_yread, bar_z[kStages], bar_s[kStages], bar_p[kStages], bar_o[kStages], bar_up[kStages],
        bar_staged[kStages], bar_u, bar_o2, bar_scaled, bar_parts, bar_zero;
    uint32_t tmem;
};

template <int D>
struct __align__(1024) SumSmem {
    uint8_t lo[kTile * D * 2], mid[kStages][kTile * D * 2];
    uint8_t y[kStages][kTile * D * 2];  // Y; then the high part
    uint8_t z[kStages][kTile * D * 2];
    uint64_t bar_load[kStages], bar_up[kStages], bar_parts[kStages], bar_lo;
    uint32_t tmem;
};

__device__ __forceinline__ void report(int32_t *err, int code)
{
    if (err != nullptr) atomicCAS(err, 0, code);
}

// Barriers and how far their two sides can be apart: a waiter must look before
// the phase after the next can complete.  Where the two chains of products
// could run ahead of a waiter (S, the state's update, the staged output) there
// is a barrier per stage: its next phase needs the stage's next load, and that
// needs the waiter's own step.  Everywhere else the next phase already needs
// the waiter.
// A wait that gives up reports, and the thread's later waits give up at once.
// A thread that loads asks for no more then, nor where its last copy into the
// same place has not landed, whose barrier still counts that one (others gave
// up on it).  What a thread has in flight it waits for at the end, a whole
// limit again; products are in order, and one that gave up issues a tile's only
// after polls that take longer than they do.
struct Waiter {
    int32_t *err;
    uint32_t limit;
    __device__ __forceinline__ void operator()(uint64_t *bar, uint32_t parity, int code)
    {
        if (!mbar_wait(bar, parity & 1, limit)) {
            report(err, code);
            limit = kGivenUp;
        }
    }
    __device__ __forceinline__ bool given_up() const { return limit == kGivenUp; }
    __device__ __forceinline__ bool may_load(uint64_t *bar, uint32_t parity) const
    {
        return !given_up() && mbar_test(bar, parity & 1);
    }
    __device__ __forceinline__ void last(uint64_t *bar, uint32_t parity, int code)
    {
        if (!mbar_wait(bar, parity & 1, kWait)) report(err, code);
    }
};

__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&p);
}

// two fp32 products in one instruction
__device__ __forceinline__ void mul2(float &x0, float &x1, float a0, float a1)
{
    asm("{\n\t.reg .b64 u, v;\n\tmov.b64 u, {%0, %1};\n\tmov.b64 v, {%2, %3};\n\t"
        "mul.rn.f32x2 u, u, v;\n\tmov.b64 {%0, %1}, u;\n\t}"
        : "+f"(x0), "+f"(x1)
        : "f"(a0), "f"(a1));
}
// pairs of bf16, each operation rounded once to bf16
__device__ __forceinline__ uint32_t bf_mul(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t bf_fma(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t bf_neg(uint32_t a) { return a ^ 0x80008000u; }

// generic-proxy writes of a warp (shared or tensor memory) handed to the issuer
__device__ __forceinline__ void hand_over(uint64_t *bar)
{
    fence_proxy_async_smem();
    tc_fence_before_sync();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// A and B K-major over K = D
template <int D>
__device__ __forceinline__ void mma_scores(uint32_t d, const uint8_t *a, const uint8_t *b)
{
    constexpr uint32_t id = idesc_bf16_f32(128, 128, false, false);
#pragma unroll
    for (int kk = 0; kk < D / 16; kk++) {
        const uint32_t off = (kk >> 2) * kBlk + (kk & 3) * 32;
        umma_bf16(d, desc_sw128(smem_u32(a) + off, 16, 1024), desc_sw128(smem_u32(b) + off, 16, 1024), id, kk > 0);
    }
}

// X [128 x D] K-major times the state operand [D x D], rows = K
template <int D>
__device__ __forceinline__ void mma_state_read(uint32_t d, const uint8_t *x, const uint8_t *u)
{
    constexpr uint32_t id = idesc_bf16_f32(128, D, false, true);
#pragma unroll
    for (int kk = 0; kk < D / 16; kk++)
        umma_bf16(d, desc_sw128(smem_u32(x) + (kk >> 2) * kBlk + (kk & 3) * 32, 16, 1024),
                  desc_sw128(smem_u32(u) + kk * 2048, (uint32_t)D * 128, 1024), id, kk > 0);
}

// O += P (tensor memory) times Z [128 x D], rows = K
template <int D>
__device__ __forceinline__ void mma_pz(uint32_t d, uint32_t p, const uint8_t *z)
{
    constexpr uint32_t id = idesc_bf16_f32(128, D, false, true);
#pragma unroll
    for (int kk = 0; kk < kTile / 16; kk++)
        umma_bf16_tmem_a(d, p + kk * 8, desc_sw128(smem_u32(z) + kk * 2048, kBlk, 1024), id, 1u);
}

// U += part^T Z: M = D (padded to 128 rows: for D = 64 the second block of A
// is whatever follows it in shared memory, rows of U nobody reads)
template <int D>
__device__ __forceinline__ void mma_state_add(uint32_t u, const uint8_t *part, const uint8_t *z, bool fresh)
{
    constexpr uint32_t id = idesc_bf16_f32(128, D, true, true);
#pragma unroll
    for (int kk = 0; kk < kTile / 16; kk++)
        umma_bf16(u, desc_sw128(smem_u32(part) + kk * 2048, kBlk, 1024),
                  desc_sw128(smem_u32(z) + kk * 2048, kBlk, 1024), id, (kk > 0 || !fresh) ? 1u : 0u);
}

template <int D>
__device__ __forceinline__ void load_tile(uint8_t *dst, const CUtensorMap *map, uint64_t *bar, int t0, int bh)
{
#pragma unroll
    for (int c = 0; c < D / 64; c++) tma_load_3d(dst + c * kBlk, map, bar, c * 64, t0, bh);
}

__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}
__device__ __forceinline__ void sts128(uint32_t a, const uint4 &v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Half hb (D / 2 columns) of row r of a 128-byte-swizzled tile: its piece c
// (8 columns, 16 bytes) is at (tile + half_row) ^ (c << 4), the tile's address
// being a multiple of 1024.
template <int D>
__device__ __forceinline__ uint32_t half_row(int r, int hb)
{
    return D == 128 ? hb * kBlk + sw128_offset(r, 0) : sw128_offset(r, hb * 4);
}

// Eight columns of u y in bf16 parts.
//
// Two parts without leaving bf16: with w = wh + wl (16 bits), hi = y wh rounded
// and y wh - hi is exact in bf16 (the error of a rounded product fits its own
// precision), so mid = y wl + (y wh - hi) is one more rounding, 2^-17 of the
// value: three operations on pairs.
__device__ __forceinline__ void split2(const uint4 &y, uint32_t wh2, uint32_t wl2, uint4 &hi, uint4 &mid)
{
#pragma unroll
    for (int e = 0; e < 4; e++) {
        const uint32_t v = reinterpret_cast<const uint32_t *>(&y)[e], p = bf_mul(v, wh2);
        reinterpret_cast<uint32_t *>(&hi)[e] = p;
        reinterpret_cast<uint32_t *>(&mid)[e] = bf_fma(v, wl2, bf_fma(v, wh2, bf_neg(p)));
    }
}

// Three parts (24 bits) from the fp32 product.
__device__ __forceinline__ void split3(const uint4 &y, float w, uint4 (&part)[3])
{
#pragma unroll
    for (int e = 0; e < 4; e++) {
        const float2 f = __bfloat1622float2(reinterpret_cast<const __nv_bfloat162 *>(&y)[e]);
        float a = f.x, b = f.y;
        mul2(a, b, w, w);
#pragma unroll
        for (int p = 0; p < 3; p++) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
            reinterpret_cast<__nv_bfloat162 *>(&part[p])[e] = h;
            const float2 g = __bfloat1622float2(h);
            a -= g.x;
            b -= g.y;
        }
    }
}

// Columns [0, 16) of row r (the warp's rows are its lanes') of an fp32 matrix of
// `rows` rows with stride `ld`.  Four lanes read a row's 64 bytes together and
// pass the pieces on, so that a load touches 8 lines instead of 32 (1024 prompts
// of 100 tokens at D = 128 from a state: 68.2 us without, 66.4 so; at D = 64, half
// a row, 41.4 and 44.2).
__device__ __forceinline__ void load_row16(const float *m, int ld, int r, int rows, float (&x)[16])
{
    const int g = r & 3;
#pragma unroll
    for (int j = 0; j < 4; j++)
        *reinterpret_cast<float4 *>(&x[4 * j]) =
            r < rows ? *reinterpret_cast<const float4 *>(m + ((r & ~3) + j) * ld + 4 * g) : make_float4(0.f, 0.f, 0.f, 0.f);
    // the 4 x 4 pieces transposed over the four lanes: odd and even ones, then pairs
#pragma unroll
    for (int step = 1; step < 4; step *= 2) {
        const bool up = g & step;
#pragma unroll
        for (int j = 0; j < 4; j++) {
            if (j & step) continue;
#pragma unroll
            for (int e = 0; e < 4; e++) {
                float &low = x[4 * j + e], &high = x[4 * (j + step) + e];
                const float got = __shfl_xor_sync(0xffffffffu, up ? low : high, step);
                low = up ? got : low;
                high = up ? high : got;
            }
        }
    }
}

// a tile's rows of `base`, d columns each, towards L2
__device__ __forceinline__ void prefetch_tile(const void *base, int d, int t0, int bh, int T)
{
    bulk_prefetch_l2((const uint8_t *)base + ((long long)bh * T + t0) * d * 2, min(kTile, T - t0) * d * 2);
}

// half hb of row r of a tile to zero
template <int D>
__device__ __forceinline__ void zero_row(const uint8_t *t, int r, int hb)
{
    const uint32_t a = smem_u32(t) + half_row<D>(r, hb);
#pragma unroll
    for (int c = 0; c < D / 16; c++) sts128(a ^ (c << 4), make_uint4(0, 0, 0, 0));
}

// the segment's tokens [lo, hi) of a sequence of `len`
__device__ __forceinline__ void segment(int seg, int seg_tiles, int len, int *lo, int *hi)
{
    const long long a = (long long)seg * seg_tiles * kTile, b = a + (long long)seg_tiles * kTile;
    *lo = (int)(a < len ? a : len);
    *hi = (int)(b < len ? b : len);
}

template <int D>
__global__ void __launch_bounds__(kWalkThreads, 1)
linattn_walk_kernel(const __grid_constant__ LinWalk W, const __grid_constant__ WalkMaps M)
{
    extern __shared__ uint8_t smem_raw[];
    WalkSmem<D> &s = *reinterpret_cast<WalkSmem<D> *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int bh = blockIdx.y, b = bh / W.H;
    const LinJob &J = W.job[blockIdx.z];
    int len = lin_length(W.lens, b, W.T);
    grid_launch_dependents();  // a state pass behind these walks takes the SMs that they leave
    if (len < 0) {
        if (tid == 0) report(W.device_error, LLA_DEVERR_BAD_LENGTH);
        len = 0;
    }
    int lo, hi;
    segment(blockIdx.x, W.seg_tiles, len, &lo, &hi);
    const int tiles = (hi - lo + kTile - 1) / kTile;
    const float *init = J.init == nullptr ? nullptr : J.init + bh * J.init_bh + blockIdx.x * J.init_seg;
    if (tiles == 0) {
        grid_dependency_wait();  // what comes after this kernel counts on the ones before it too
        return;
    }
    const bool rev = J.rev != 0;
    // token range of the n-th tile of the walk
    auto tile_start = [&](int n) { return lo + (rev ? tiles - 1 - n : n) * kTile; };
    auto tile_rows = [&](int n) { return min(kTile, hi - tile_start(n)); };
    auto load_x = [&](int n) {
        mbar_arrive_expect_tx(&s.bar_x, kTile * D * 2);
        load_tile<D>(s.x, &M.x[blockIdx.z], &s.bar_x, tile_start(n), bh);
    };
    auto load_y = [&](int n) {
        mbar_arrive_expect_tx(&s.bar_y, kTile * D * 2);
        load_tile<D>(s.y, &M.y[blockIdx.z], &s.bar_y, tile_start(n), bh);
    };
    auto load_z = [&](int n) {
        mbar_arrive_expect_tx(&s.bar_z[n % kStages], kTile * D * 2);
        load_tile<D>(s.z[n % kStages], &M.z[blockIdx.z], &s.bar_z[n % kStages], tile_start(n), bh);
    };
    // the two loading threads ask for the first tiles at once, while the CTA gets ready
    if (tid == kLoadThread) {
        mbar_init(&s.bar_x, 1);
        mbar_init(&s.bar_y, 1);
        fence_mbar_init();
        fence_proxy_async_smem();
        load_y(0);
        load_x(0);
    }
    if (tid == kStoreThread) {
        for (int i = 0; i < kStages; i++) mbar_init(&s.bar_z[i], 1);
        fence_mbar_init();
        fence_proxy_async_smem();
        for (int n = 0; n < min(kStages, tiles); n++) load_z(n);
        tma_prefetch_map(&M.out[blockIdx.z]);
    }
    const float ld = W.log_decay[bh % W.H];
    for (int e = tid; e <= kTile; e += kWalkThreads) s.pw[e] = decay_pow(ld, e);
    if (tid < 32) s.cf[tid] = decay_pow(ld, rev ? tid : 31 - tid);
    if (tid < 64) s.diag[tid] = tid < 32 ? 0.f : decay_pow(ld, tid - 32);
    if (tid == 0) {
        for (int i = 0; i < kStages; i++) {
            mbar_init(&s.bar_s[i], 1);
            mbar_init(&s.bar_p[i], kRowWarps);
            mbar_init(&s.bar_o[i], 1);
            mbar_init(&s.bar_up[i], 1);
            mbar_init(&s.bar_staged[i], kRowWarps);
        }
        mbar_init(&s.bar_yread, kStateWarps);
        mbar_init(&s.bar_u, kStateWarps);
        mbar_init(&s.bar_o2, 1);
        mbar_init(&s.bar_scaled, kStateWarps);
        mbar_init(&s.bar_parts, kStateWarps);
        mbar_init(&s.bar_zero, kStateWarps);
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(&s.tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    // columns: S [0,128), O of even and of odd tiles, U.  P of a tile takes the first 64 columns of the
    // other O, between that one's way out and the next tile's read-out
    const uint32_t tm_s = s.tmem, tm_o0 = tm_s + 128, tm_u = tm_o0 + 2 * D;
    auto tm_o = [&](int n) { return tm_o0 + (uint32_t)(n & 1) * D; };
    Waiter wait{W.device_error, kWait};
    // the output tile goes out by a bulk copy, clipped at T; one that ends before T is stored row by row
    auto store_direct = [&](int n) { return tile_rows(n) < kTile && tile_start(n) + tile_rows(n) != W.T; };

    if (warp < kRowWarps) {
        // ---- scores to P, outputs; two threads per row i, each half of the columns
        const int quad = warp & 3, half = warp >> 2;
        const int i = quad * 32 + lane;
        const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
        auto make_p = [&](int n) {
            const uint32_t tm = tm_s + lane_off;
            wait(&s.bar_s[n % kStages], n / kStages, LLA_DEVERR_SYNC_TIMEOUT);
            tc_fence_after_sync();
            // every other 32-column block of S to 16 packed columns of P
            float pk[2][16];  // packed pairs, as bits
#pragma unroll
            for (int u = 0; u < 2; u++) {
                const int c32 = half + 2 * u, j0 = c32 * 32;
                if (rev ? c32 < quad : c32 > quad) {  // the whole block is masked
#pragma unroll
                    for (int e = 0; e < 16; e++) pk[u][e] = 0.f;
                    continue;
                }
                float x[2][16];
                tmem_ld16(tm + j0, x[0]);
                tmem_ld16(tm + j0 + 16, x[1]);
                tmem_ld_wait();
                if (c32 == quad) {
                    const float *f = s.diag + 32 + (rev ? -lane : lane);
#pragma unroll
                    for (int c = 0; c < 32; c += 2) {
                        const float f0 = rev ? f[c] : f[-c], f1 = rev ? f[c + 1] : f[-c - 1];
                        mul2(x[c / 16][c % 16], x[c / 16][c % 16 + 1], f0, f1);
                    }
                } else {
                    const float rowf = s.pw[rev ? j0 - i : i - j0 - 31];
#pragma unroll
                    for (int c = 0; c < 32; c += 4) {
                        float4 f = *reinterpret_cast<const float4 *>(&s.cf[c]);
                        mul2(f.x, f.y, rowf, rowf);
                        mul2(f.z, f.w, rowf, rowf);
                        mul2(x[c / 16][c % 16], x[c / 16][c % 16 + 1], f.x, f.y);
                        mul2(x[c / 16][c % 16 + 2], x[c / 16][c % 16 + 3], f.z, f.w);
                    }
                }
#pragma unroll
                for (int c = 0; c < 32; c += 2)
                    pk[u][c / 2] = __uint_as_float(pack_bf16(x[c / 16][c % 16], x[c / 16][c % 16 + 1]));
            }
            // P goes over columns of the last tile's O that the other warp of these rows takes out
            tc_fence_before_sync();
            asm volatile("bar.sync %0, 64;" ::"r"(1 + quad) : "memory");
            tc_fence_after_sync();
#pragma unroll
            for (int u = 0; u < 2; u++) tmem_st16(tm_o(n + 1) + lane_off + (half + 2 * u) * 16, pk[u]);
            tmem_st_wait();
            hand_over(&s.bar_p[n % kStages]);
        };
        make_p(0);
        for (int n = 0; n < tiles; n++) {
            const int st = n % kStages;
            wait(&s.bar_o[st], n / kStages, LLA_DEVERR_SYNC_TIMEOUT);
            // Z's place takes the output tile once its last reader, the state's update, is done: of the
            // inputs it is the one needed last in the next tile but one
            if (n + 1 < tiles) wait(&s.bar_up[st], n / kStages, LLA_DEVERR_SYNC_TIMEOUT);
            tc_fence_after_sync();
            const uint32_t tm_mine = tm_o(n) + lane_off + half * (D / 2);
            const uint32_t stage = smem_u32(s.z[st]) + half_row<D>(i, half);
#pragma unroll
            for (int c0 = 0; c0 < D / 2; c0 += 32) {
                float x[2][16];
                tmem_ld16(tm_mine + c0, x[0]);
                tmem_ld16(tm_mine + c0 + 16, x[1]);
                tmem_ld_wait();
                uint4 o[4];
#pragma unroll
                for (int c = 0; c < 32; c += 2)
                    reinterpret_cast<uint32_t *>(o)[c / 2] = pack_bf16(x[c / 16][c % 16], x[c / 16][c % 16 + 1]);
#pragma unroll
                for (int e = 0; e < 4; e++) sts128(stage ^ ((c0 / 8 + e) << 4), o[e]);
            }
            if (store_direct(n) && i < tile_rows(n)) {  // the thread's own pieces back
                __nv_bfloat16 *dst = (__nv_bfloat16 *)J.out + ((long long)bh * W.T + tile_start(n) + i) * J.dz;
#pragma unroll 1
                for (int c = half * (D / 2); c < min(J.dz, (half + 1) * (D / 2)); c += 8)
                    *reinterpret_cast<uint4 *>(dst + c) = lds128(stage ^ ((c % (D / 2)) << 1));
            }
            hand_over(&s.bar_staged[st]);
            if (n + 1 < tiles) make_p(n + 1);
        }
    } else if (warp < kRowWarps + kStateWarps) {
        // ---- the state; thread = row r of U (and of the token tile), half hb of its columns
        const int r = (warp & 3) * 32 + lane, hb = (warp - kRowWarps) >> 2;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const bool has_u = (warp & 3) * 32 < D;  // whole warps
        constexpr int kHalf = D / 2;
        const uint32_t tm_mine = tm_u + lane_off + hb * kHalf;
        const uint32_t mine = half_row<D>(r, hb);
        grid_dependency_wait();  // all that a kernel before this one may have made are the states
        if (has_u) {
#pragma unroll
            for (int c0 = 0; c0 < kHalf; c0 += 16) {
                float x[16];
                const int c = hb * kHalf + c0;
#pragma unroll
                for (int e = 0; e < 16; e++) x[e] = 0.f;
                if (init != nullptr && c < J.dz) {  // dx and dz are multiples of 16
                    if (D == 128 && !J.init_t) {
                        load_row16(init + c, J.dz, r, J.dx, x);
                    } else if (r < J.dx && J.init_t) {
#pragma unroll
                        for (int e = 0; e < 16; e++) x[e] = init[(c + e) * J.dx + r];
                    } else if (r < J.dx) {
#pragma unroll
                        for (int e = 0; e < 16; e += 4)
                            *reinterpret_cast<float4 *>(&x[e]) = *reinterpret_cast<const float4 *>(init + r * J.dz + c + e);
                    }
                }
                tmem_st16(tm_mine + c0, x);
            }
            tmem_st_wait();
        }
        for (int n = 0; n < tiles; n++) {
            const int st = n % kStages, rows = tile_rows(n);
            if (rows < kTile) {  // rows behind the sequence count as zeros, whatever they hold
                wait(&s.bar_y, n, LLA_DEVERR_COPY_TIMEOUT);
                wait(&s.bar_z[st], n / kStages, LLA_DEVERR_COPY_TIMEOUT);
                if (r >= rows) {
                    zero_row<D>(s.y, r, hb);
                    zero_row<D>(s.z[st], r, hb);
                }
                hand_over(&s.bar_zero);
            }
            // the thread's part of Y, while the last tile's update runs
            uint4 y[D / 16];
            wait(&s.bar_y, n, LLA_DEVERR_COPY_TIMEOUT);
#pragma unroll
            for (int c = 0; c < D / 16; c++) y[c] = lds128((smem_u32(s.y) + mine) ^ (c << 4));
            if (n > 0) {
                wait(&s.bar_up[(n - 1) % kStages], (n - 1) / kStages, LLA_DEVERR_SYNC_TIMEOUT);
                tc_fence_after_sync();
            }
            // U to its bf16 operand, and decayed over this tile
            if (has_u) {
                const float an = s.pw[rows];
#pragma unroll
                for (int c0 = 0; c0 < kHalf; c0 += 32) {
                    float x[2][16];
                    tmem_ld16(tm_mine + c0, x[0]);
                    tmem_ld16(tm_mine + c0 + 16, x[1]);
                    tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        uint4 pk;
#pragma unroll
                        for (int c = 0; c < 8; c += 2) {
                            float &a = x[e / 2][(8 * e + c) % 16], &b = x[e / 2][(8 * e + c) % 16 + 1];
                            reinterpret_cast<uint32_t *>(&pk)[c / 2] = pack_bf16(a, b);
                            mul2(a, b, an, an);
                        }
                        sts128((smem_u32(s.u) + mine) ^ ((c0 / 8 + e) << 4), pk);
                    }
                    tmem_st16(tm_mine + c0, x[0]);
                    tmem_st16(tm_mine + c0 + 16, x[1]);
                }
                tmem_st_wait();
            }
            hand_over(&s.bar_u);
            // u y in parts (nothing reads the last tile's state)
            if (n + 1 < tiles) {
                const float w = s.pw[r < rows ? (rev ? r + 1 : rows - 1 - r) : 0];
                const float wh = __bfloat162float(__float2bfloat16_rn(w));
                const uint32_t wh2 = pack_bf16(wh, wh), wl2 = pack_bf16(w - wh, w - wh);
#pragma unroll
                for (int c = 0; c < D / 16; c++) {
                    uint4 hi, mid;
                    split2(y[c], wh2, wl2, hi, mid);
                    sts128((smem_u32(s.hi) + mine) ^ (c << 4), hi);
                    sts128((smem_u32(s.mid) + mine) ^ (c << 4), mid);
                }
                hand_over(&s.bar_parts);
                // Y's place is given up only here, behind stores of what was read from it: an arrival does not
                // wait for reads under way, and the next copy is short
                if (lane == 0) mbar_arrive(&s.bar_yread);
            }
            wait(&s.bar_o2, n, LLA_DEVERR_SYNC_TIMEOUT);
            // the read-out times its row's decay; P Z is added to it
            tc_fence_after_sync();
            const float wi = r < rows ? s.pw[rev ? rows - 1 - r : r + 1] : 0.f;
#pragma unroll
            for (int c0 = 0; c0 < kHalf; c0 += 32) {
                float x[2][16];
                const uint32_t tm = tm_o(n) + lane_off + hb * kHalf + c0;
                tmem_ld16(tm, x[0]);
                tmem_ld16(tm + 16, x[1]);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < 32; c += 2) mul2(x[c / 16][c % 16], x[c / 16][c % 16 + 1], wi, wi);
                tmem_st16(tm, x[0]);
                tmem_st16(tm + 16, x[1]);
            }
            tmem_st_wait();
            hand_over(&s.bar_scaled);
        }
    } else {
        const int role = warp - kRowWarps - kStateWarps;
        if (lane != 0 || (W.withhold && role == 1)) {  // withheld: nothing is left in flight, the waits on S run out
        } else if (role == 0) {  // ---- loads of x and y, one tile ahead (z: with the output)
            // one place each: the next tile's rows are brought to L2 meanwhile, so that their load is short
            auto ahead = [&](const void *base, int n) {
                if (n < tiles) prefetch_tile(base, J.dx, tile_start(n), bh, W.T);
            };
            int nx = 0, ny = 0;  // the last tiles asked for
            for (int n = 0; n < tiles; n++) {
                // y: S has been formed and the state warps have theirs; x: the state has been read out too
                if (n > 0) {
                    wait(&s.bar_s[(n - 1) % kStages], (n - 1) / kStages, LLA_DEVERR_SYNC_TIMEOUT);
                    wait(&s.bar_yread, n - 1, LLA_DEVERR_SYNC_TIMEOUT);
                    if (!wait.may_load(&s.bar_y, n - 1)) break;
                    load_y(ny = n);
                }
                ahead(J.x, n + 1);
                ahead(J.y, n + 1);
                if (n > 0) {
                    wait(&s.bar_o2, n - 1, LLA_DEVERR_SYNC_TIMEOUT);
                    if (!wait.may_load(&s.bar_x, n - 1)) break;
                    load_x(nx = n);
                }
            }
            // no copy is in flight when the CTA ends
            wait.last(&s.bar_x, nx, LLA_DEVERR_COPY_TIMEOUT);
            wait.last(&s.bar_y, ny, LLA_DEVERR_COPY_TIMEOUT);
        } else if (role == 1) {  // ---- the scores' products: S of the next tile and P Z of this one, as they can go
            auto scores = [&](int n) {
                tc_fence_after_sync();
                mma_scores<D>(tm_s, s.x, s.y);
                umma_commit(&s.bar_s[n % kStages]);
            };
            // S of tile n: its inputs are there (a short tile's rows behind the sequence as zeros; one tile
            // of a walk at most is short), and the last S has become P
            auto scores_ready = [&](int n) {
                return mbar_test(&s.bar_x, n & 1) && mbar_test(&s.bar_y, n & 1) &&
                       (tile_rows(n) == kTile || mbar_test(&s.bar_zero, 0)) &&
                       (n == 0 || mbar_test(&s.bar_p[(n - 1) % kStages], ((n - 1) / kStages) & 1));
            };
            for (int n = -1; n < tiles; n++) {
                bool next = n + 1 < tiles, pz = n >= 0;
                for (uint32_t polls = 0; next || pz; polls++) {
                    const bool give_up = polls >= (wait.limit == kWait ? kIssuerSpin : kGivenUp);
                    if (give_up) {
                        report(W.device_error, LLA_DEVERR_SYNC_TIMEOUT);
                        wait.limit = kGivenUp;
                    }
                    if (polls > 0) __nanosleep(32);  // its polls take issue slots from the working warps
                    if (pz && (give_up || (mbar_test(&s.bar_scaled, n & 1) &&
                                           mbar_test(&s.bar_p[n % kStages], (n / kStages) & 1) &&
                                           mbar_test(&s.bar_z[n % kStages], (n / kStages) & 1)))) {
                        tc_fence_after_sync();
                        mma_pz<D>(tm_o(n), tm_o(n + 1), s.z[n % kStages]);
                        umma_commit(&s.bar_o[n % kStages]);
                        pz = false;
                    }
                    if (next && (give_up || scores_ready(n + 1))) {
                        scores(n + 1);
                        next = false;
                    }
                }
            }
            // every product has completed when the tensor memory is freed
            wait.last(&s.bar_o[(tiles - 1) % kStages], (tiles - 1) / kStages, LLA_DEVERR_SYNC_TIMEOUT);
        } else if (role == 2) {  // ---- output tiles on their way out, and loads of z into the places they leave
            int asked = min(kStages, tiles);
            for (int n = 0; n < tiles; n++) {
                const int st = n % kStages;
                wait(&s.bar_staged[st], n / kStages, LLA_DEVERR_SYNC_TIMEOUT);
                if (!store_direct(n)) {
                    for (int c = 0; c < D / 64 && c * 64 < J.dz; c++)
                        tma_store_3d(&M.out[blockIdx.z], s.z[st] + c * kBlk, c * 64, tile_start(n), bh);
                    tma_store_commit();
                    tma_store_wait_read();
                }
                if (n + kStages < tiles) {
                    if (!wait.may_load(&s.bar_z[st], n / kStages)) break;
                    load_z(n + kStages);
                    asked = n + kStages + 1;
                }
            }
            for (int n = max(0, asked - kStages); n < asked; n++)
                wait.last(&s.bar_z[n % kStages], n / kStages, LLA_DEVERR_COPY_TIMEOUT);
        } else {  // ---- the state's products: its read-out, then its update
            for (int n = 0; n < tiles; n++) {
                const int st = n % kStages;
                wait(&s.bar_x, n, LLA_DEVERR_COPY_TIMEOUT);
                // this O held the last tile's P
                if (n > 0) wait(&s.bar_o[(n - 1) % kStages], (n - 1) / kStages, LLA_DEVERR_SYNC_TIMEOUT);
                wait(&s.bar_u, n, LLA_DEVERR_SYNC_TIMEOUT);
                tc_fence_after_sync();
                mma_state_read<D>(tm_o(n), s.x, s.u);
                umma_commit(&s.bar_o2);
                if (n + 1 == tiles) break;
                wait(&s.bar_z[st], n / kStages, LLA_DEVERR_COPY_TIMEOUT);
                wait(&s.bar_parts, n, LLA_DEVERR_SYNC_TIMEOUT);
                tc_fence_after_sync();
                mma_state_add<D>(tm_u, s.hi, s.z[st], false);
                mma_state_add<D>(tm_u, s.mid, s.z[st], false);
                umma_commit(&s.bar_up[st]);
            }
            // every product has completed when the tensor memory is freed
            wait.last(&s.bar_o2, tiles - 1, LLA_DEVERR_SYNC_TIMEOUT);
        }
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tm_s, 512);
}

// A segment's own sum: u y against z over its tokens, u the powers of the
// decay to the segment's far edge, so that nothing is rescaled on the way.
//
// u y goes in three bf16 parts (24 bits).  The tensor cores do not round their
// fp32 accumulator to nearest, and over hundreds of products the bias shows
// (8e-6 of the state after 29 tiles); so every tile has a fresh accumulator,
// the small middle part first, and the tiles are added up in registers (the
// same state: 4e-7).
//
// A tile takes 2.1 us at D = 128, bound by shared memory: three products read
// both operands there (192 KB), the split reads 32 KB and writes 96, the copies
// write 64, about 3000 of its 3900 cycles.  Over whole sequences the pass runs
// behind the walks, on SMs that they do not take or have left (gradients of 2 x
// 16 heads of 8192 tokens: 6 us for it, 48 as a kernel of its own before them).
template <int D>
__global__ void __launch_bounds__(kSumThreads, 1)
linattn_sum_kernel(const __grid_constant__ LinWalk W, const __grid_constant__ WalkMaps M)
{
    extern __shared__ uint8_t smem_raw[];
    SumSmem<D> &s = *reinterpret_cast<SumSmem<D> *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    grid_launch_dependents();  // the scan's CTAs are small: they start beside these and wait
    const int bh = blockIdx.y, b = bh / W.H;
    const LinJob &J = W.job[blockIdx.z];
    const int len = lin_length(W.lens, b, W.T);
    if (len < 0) {
        if (tid == 0) report(W.device_error, LLA_DEVERR_BAD_LENGTH);
        grid_dependency_wait();  // what comes after this kernel counts on the one before it too
        return;
    }
    int lo, hi;
    segment(blockIdx.x, W.seg_tiles, len, &lo, &hi);
    const int tiles = (hi - lo + kTile - 1) / kTile;
    const int dx = J.dx, dz = J.dz;  // both at most D
    float *fin = J.final_ + ((long long)bh * W.nseg + blockIdx.x) * dx * dz;
    const float *init = J.init == nullptr ? nullptr : J.init + bh * J.init_bh;
    if (tiles == 0) {
        grid_dependency_wait();
        for (int e = tid; e < dx * dz; e += kSumThreads) fin[e] = init == nullptr ? 0.f : init[e];
        return;
    }
    const bool rev = J.rev != 0;
    auto load = [&](int n) {
        const int st = n % kStages;
        mbar_arrive_expect_tx(&s.bar_load[st], 2 * kTile * D * 2);
        load_tile<D>(s.y[st], &M.y[blockIdx.z], &s.bar_load[st], lo + n * kTile, bh);
        load_tile<D>(s.z[st], &M.z[blockIdx.z], &s.bar_load[st], lo + n * kTile, bh);
    };
    if (tid == kSumWarps * 32) {  // the loading thread: the first tiles at once, while the CTA gets ready
        for (int i = 0; i < kStages; i++) mbar_init(&s.bar_load[i], 1);
        fence_mbar_init();
        fence_proxy_async_smem();
        for (int n = 0; n < min(kStages, tiles); n++) load(n);
    }
    const float ld = W.log_decay[bh % W.H];
    if (tid == 0) {
        for (int i = 0; i < kStages; i++) mbar_init(&s.bar_up[i], 1);
        mbar_init(&s.bar_lo, kSumWarps);
        for (int i = 0; i < kStages; i++) mbar_init(&s.bar_parts[i], kSumWarps);
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(&s.tmem, 256);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tm_u = s.tmem;
    Waiter wait{W.device_error, kWait};
    if (warp < kSumWarps) {
        constexpr int kPieces = D / 32;  // of 8 columns: a quarter of the row
        const int r = (warp & 3) * 32 + lane, quarter = warp >> 2;
        const uint32_t mine = half_row<D>(r, quarter >> 1) ^ ((quarter & 1) * kPieces << 4);
        const bool has_u = (warp & 3) * 32 < D;  // whole warps
        float sum[D / 64][16];  // D / 4 columns
#pragma unroll
        for (int k = 0; k < D / 64; k++)
#pragma unroll
            for (int e = 0; e < 16; e++) sum[k][e] = 0.f;
        auto add_tile = [&](int n) {  // the thread's quarter of its row of tile n's accumulator
            if (!has_u) return;
            tc_fence_after_sync();
            float x[D / 64][16];
#pragma unroll
            for (int k = 0; k < D / 64; k++)
                tmem_ld16(tm_u + (n & 1) * 128 + ((uint32_t)((warp & 3) * 32) << 16) + quarter * (D / 4) + 16 * k, x[k]);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < D / 64; k++)
#pragma unroll
                for (int e = 0; e < 16; e++) sum[k][e] += x[k][e];
        };
        for (int n = 0; n < tiles; n++) {
            const int st = n % kStages, t = lo + n * kTile + r;
            const bool counts = t < hi;
            const float w = decay_pow(ld, counts ? (rev ? t - lo + 1 : hi - 1 - t) : 0);
            wait(&s.bar_load[st], n / kStages, LLA_DEVERR_COPY_TIMEOUT);
            const uint32_t y = smem_u32(s.y[st]) + mine, z = smem_u32(s.z[st]) + mine;
            uint4 low[kPieces];
#pragma unroll
            for (int c = 0; c < kPieces; c++) {
                uint4 part[3];
                // a row behind the sequence counts as zeros, whatever it holds
                split3(counts ? lds128(y ^ (c << 4)) : make_uint4(0, 0, 0, 0), w, part);
                sts128(y ^ (c << 4), part[0]);
                if (!counts) sts128(z ^ (c << 4), make_uint4(0, 0, 0, 0));
                sts128((smem_u32(s.mid[st]) + mine) ^ (c << 4), part[1]);
                low[c] = part[2];
            }
            // the first two products go out behind the last tile's; the low part waits for its place
            hand_over(&s.bar_parts[st]);
            if (n > 0) wait(&s.bar_up[(n - 1) % kStages], (n - 1) / kStages, LLA_DEVERR_SYNC_TIMEOUT);
#pragma unroll
            for (int c = 0; c < kPieces; c++) sts128((smem_u32(s.lo) + mine) ^ (c << 4), low[c]);
            hand_over(&s.bar_lo);
            if (n > 0) add_tile(n - 1);  // before this warp's next parts, which its accumulator's next tile needs
        }
        wait(&s.bar_up[(tiles - 1) % kStages], (tiles - 1) / kStages, LLA_DEVERR_SYNC_TIMEOUT);
        add_tile(tiles - 1);
        // walks before this pass may still read a state that is written here
        grid_dependency_wait();
        const float all = decay_pow(ld, hi - lo);
        // two lanes take a row's 32 bytes together: 16 of a row from each lane would go out as half sectors
        const bool odd = lane & 1;
#pragma unroll
        for (int k = 0; k < D / 64; k++) {
            const int c0 = quarter * (D / 4) + 16 * k;
            if (c0 >= dz) break;  // dx and dz are multiples of 16
#pragma unroll
            for (int e = 0; e < 16; e += 8) {
                float t[2][4];  // four columns of rows r & ~1 and r | 1
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float lo4 = sum[k][e + i], hi4 = sum[k][e + 4 + i];
                    const float got = __shfl_xor_sync(0xffffffffu, odd ? lo4 : hi4, 1);
                    t[0][i] = odd ? got : lo4;
                    t[1][i] = odd ? hi4 : got;
                }
                if (r < dx) {
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        const int at = ((r & ~1) + i) * dz + c0 + e + (odd ? 4 : 0);
                        float4 u = make_float4(t[i][0], t[i][1], t[i][2], t[i][3]);
                        if (init != nullptr) {
                            const float4 in = *reinterpret_cast<const float4 *>(init + at);
                            u = make_float4(fmaf(all, in.x, u.x), fmaf(all, in.y, u.y), fmaf(all, in.z, u.z), fmaf(all, in.w, u.w));
                        }
                        *reinterpret_cast<float4 *>(fin + at) = u;
                    }
                }
            }
        }
    } else if (warp == kSumWarps) {
        if (lane == 0) {
            int asked = min(kStages, tiles);
            for (int n = 0; n < tiles; n++) {
                const int st = n % kStages;
                // the tile after the next to L2: a stage is free only when its products are done
                if (n + kStages < tiles) {
                    prefetch_tile(J.y, dx, lo + (n + kStages) * kTile, bh, W.T);
                    prefetch_tile(J.z, dz, lo + (n + kStages) * kTile, bh, W.T);
                }
                if (n >= kStages) {
                    wait(&s.bar_up[st], n / kStages - 1, LLA_DEVERR_SYNC_TIMEOUT);
                    if (!wait.may_load(&s.bar_load[st], n / kStages - 1)) break;
                    load(n);
                    asked = n + 1;
                }
            }
            for (int n = max(0, asked - kStages); n < asked; n++)
                wait.last(&s.bar_load[n % kStages], n / kStages, LLA_DEVERR_COPY_TIMEOUT);
        }
    } else if (lane == 0 && !W.withhold) {  // withheld: nothing is left in flight, the waits on bar_up run out
        for (int n = 0; n < tiles; n++) {
            const int st = n % kStages;
            wait(&s.bar_parts[st], n / kStages, LLA_DEVERR_SYNC_TIMEOUT);
            tc_fence_after_sync();
            const uint32_t acc = tm_u + (n & 1) * 128;
            mma_state_add<D>(acc, s.mid[st], s.z[st], true);
            mma_state_add<D>(acc, s.y[st], s.z[st], false);
            wait(&s.bar_lo, n, LLA_DEVERR_SYNC_TIMEOUT);
            tc_fence_after_sync();
            mma_state_add<D>(acc, s.lo, s.z[st], false);
            umma_commit(&s.bar_up[st]);
        }
        wait.last(&s.bar_up[(tiles - 1) % kStages], (tiles - 1) / kStages, LLA_DEVERR_SYNC_TIMEOUT);
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tm_u, 256);
}

template <int D>
cudaError_t launch(const LinWalk &W, bool sums, bool dependent)
{
    WalkMaps M;
    const uint64_t BH = (uint64_t)W.B * W.H;
    // one map a tensor: the jobs of a call read the same ones
    struct Seen {
        const void *base;
        int d;
    } seen[4 * kLinMaxJobs];
    const CUtensorMap *made[4 * kLinMaxJobs];
    int n = 0;
    auto map = [&](CUtensorMap *m, const void *base, int d) {
        for (int i = 0; i < n; i++)
            if (seen[i].base == base && seen[i].d == d) {
                *m = *made[i];
                return true;
            }
        seen[n] = {base, d};
        made[n++] = m;
        return make_map_bf16_3d(m, base, d, W.T, BH, 64, kTile);
    };
    for (int j = 0; j < W.njobs; j++) {
        const LinJob &J = W.job[j];
        if (!map(&M.y[j], J.y, J.dx) || !map(&M.z[j], J.z, J.dz) ||
            (!sums && (!map(&M.x[j], J.x, J.dx) || !map(&M.out[j], J.out, J.dz))))
            return cudaErrorInvalidValue;
    }
    const size_t smem = (sums ? sizeof(SumSmem<D>) : sizeof(WalkSmem<D>)) + 1024;
    void (*k)(LinWalk, WalkMaps) = sums ? linattn_sum_kernel<D> : linattn_walk_kernel<D>;
    static std::atomic<uint64_t> on[2];
    cudaError_t e = allow_shared((const void *)k, smem, on[sums]);
    if (e != cudaSuccess) return e;
    return launch_kernel(k, dim3((unsigned)W.nseg, (unsigned)BH, (unsigned)W.njobs), sums ? kSumThreads : kWalkThreads,
                         smem, W.stream, dependent, W, M);
}

}  // namespace

bool linattn_tc_supported(lla_dtype dt) { return dt == LLA_BF16; }

cudaError_t linattn_tc(const LinWalk &W, bool states_only, bool dependent)
{
    return W.job[0].dx > 64 || W.job[0].dz > 64 ? launch<128>(W, states_only, dependent)
                                                : launch<64>(W, states_only, dependent);
}

}  // namespace lla
