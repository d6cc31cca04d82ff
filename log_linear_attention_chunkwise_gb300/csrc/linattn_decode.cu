// Linear attention with one decay per head, one token per sequence:
//   S = a S + k v^T,   o = q S,   a = exp(log_decay)
// on states kept in a pool, slots[b] naming the state of sequence b.
//
// Bound by the state's bytes (read and written once).  A state is cut by
// columns, 32 to a CTA (a 128-byte line of every row), so no sum crosses CTAs
// and one sequence of a few heads still spreads over the SMs; each thread
// holds its rows' pieces of four columns in registers, all loads issued at
// once, and the read-out's row sum goes over shuffles and shared memory.
// A slot that two sequences name would be a race: every CTA looks its slot up
// among all the others while its loads are in flight and leaves such a
// sequence alone.  That is 4 B bytes a CTA, which the state's 16 KB hide up to
// about a thousand sequences and not beyond: the calls with slots, against those
// without, d = 128: 1024 x 16 heads 324 us and 306, 4096 x 16 1346 and 1203,
// 16384 x 4 2152 and 1203, 65535 x 1 8639 and 1203; d = 16: 16384 x 1 93 and 17.
//
// Measured: 64 sequences of 16 heads, d = 128, the kernel 20 us for 135 MB (6.7
// TB/s), the call 25; a call for one sequence of 8 heads is the host's 15 to 20.
#include "linattn.cuh"

namespace lla {
namespace {

constexpr int kThreads = 128;

template <typename T, int DK, int CB>
__global__ void __launch_bounds__(kThreads)
linattn_decode_kernel(LinDecodeArgs A)
{
    constexpr int kLanes = CB / 4;             // threads along a row's columns
    constexpr int kRows = kThreads / kLanes;   // row groups
    constexpr int kPer = (DK + kRows - 1) / kRows;
    __shared__ float4 red[kThreads / 32][kLanes];
    const int tid = threadIdx.x, cx = tid % kLanes, ry = tid / kLanes;
    const int parts = A.dv / CB;
    const int part = blockIdx.x % parts, h = blockIdx.x / parts, b = blockIdx.y;
    const long long bh = (long long)b * A.H + h;
    // a sequence without a state of its own: its columns of out
    auto skip = [&](bool bad) {
        if (bad && tid == 0 && A.device_error != nullptr) atomicCAS(A.device_error, 0, 1 + b);
        if (A.clear_skipped && tid < kLanes)
            *reinterpret_cast<float4 *>(A.out + bh * A.dv + part * CB + 4 * tid) = make_float4(0.f, 0.f, 0.f, 0.f);
    };
    int slot = b;
    if (A.slots != nullptr) {
        slot = A.slots[b];
        if (slot < 0 || slot >= A.pool) return skip(slot >= 0);
    }
    const int col = part * CB + 4 * cx;
    float *S = A.state + ((long long)slot * A.H + h) * DK * A.dv + col;
    float4 s[kPer];
#pragma unroll
    for (int i = 0; i < kPer; i++) {
        const int r = ry + i * kRows;
        s[i] = r < DK ? *reinterpret_cast<const float4 *>(S + (long long)r * A.dv) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const float a = decay_pow(A.log_decay[h], 1);
    const T *q = (const T *)A.q + bh * DK, *k = (const T *)A.k + bh * DK, *v = (const T *)A.v + bh * A.dv + col;
    float qv[kPer], kv[kPer], vv[4];
#pragma unroll
    for (int i = 0; i < kPer; i++) {
        const int r = ry + i * kRows;
        qv[i] = r < DK ? to_f32<T>(q[r]) : 0.f;
        kv[i] = r < DK ? to_f32<T>(k[r]) : 0.f;
    }
#pragma unroll
    for (int c = 0; c < 4; c++) vv[c] = to_f32<T>(v[c]);
    if (A.slots != nullptr) {
        bool twice = false;
        for (int j = tid; j < A.B; j += kThreads) twice |= j != b && A.slots[j] == slot;
        if (__syncthreads_or(twice)) return skip(true);
    }
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kPer; i++) {
        const int r = ry + i * kRows;
        s[i].x = fmaf(kv[i], vv[0], a * s[i].x);
        s[i].y = fmaf(kv[i], vv[1], a * s[i].y);
        s[i].z = fmaf(kv[i], vv[2], a * s[i].z);
        s[i].w = fmaf(kv[i], vv[3], a * s[i].w);
        o.x = fmaf(qv[i], s[i].x, o.x);
        o.y = fmaf(qv[i], s[i].y, o.y);
        o.z = fmaf(qv[i], s[i].z, o.z);
        o.w = fmaf(qv[i], s[i].w, o.w);
        if (r < DK) *reinterpret_cast<float4 *>(S + (long long)r * A.dv) = s[i];
    }
#pragma unroll
    for (int off = 16; off >= kLanes; off >>= 1) {
        o.x += __shfl_xor_sync(0xffffffffu, o.x, off);
        o.y += __shfl_xor_sync(0xffffffffu, o.y, off);
        o.z += __shfl_xor_sync(0xffffffffu, o.z, off);
        o.w += __shfl_xor_sync(0xffffffffu, o.w, off);
    }
    if ((tid & 31) < kLanes) red[tid >> 5][cx] = o;
    __syncthreads();
    if (tid < kLanes) {
        o = red[0][tid];
#pragma unroll
        for (int w = 1; w < kThreads / 32; w++) {
            o.x += red[w][tid].x;
            o.y += red[w][tid].y;
            o.z += red[w][tid].z;
            o.w += red[w][tid].w;
        }
        *reinterpret_cast<float4 *>(A.out + bh * A.dv + part * CB + 4 * tid) = o;
    }
}

template <typename T, int CB>
void (*kernel_for(int dk))(LinDecodeArgs)
{
    switch (dk) {
    case 16: return linattn_decode_kernel<T, 16, CB>;
    case 32: return linattn_decode_kernel<T, 32, CB>;
    case 64: return linattn_decode_kernel<T, 64, CB>;
    default: return linattn_decode_kernel<T, 128, CB>;
    }
}

}  // namespace

cudaError_t linattn_decode(const LinDecodeArgs &A)
{
    const int cb = A.dv >= 32 ? 32 : 16;
    void (*k)(LinDecodeArgs);
    if (A.dt == LLA_BF16)
        k = cb == 32 ? kernel_for<__nv_bfloat16, 32>(A.dk) : kernel_for<__nv_bfloat16, 16>(A.dk);
    else
        k = cb == 32 ? kernel_for<float, 32>(A.dk) : kernel_for<float, 16>(A.dk);
    k<<<dim3((unsigned)(A.H * (A.dv / cb)), (unsigned)A.B), kThreads, 0, (cudaStream_t)A.stream>>>(A);
    return cudaPeekAtLastError();
}

}  // namespace lla
