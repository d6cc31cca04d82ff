// Internal interface of linear attention with one decay per head.
//
// Every direction is one operation on three inputs x, y, z, walked over the
// tokens with a state U (dx x dz) and a = exp(log_decay):
//   forward in time   out_i = sum_{j<=i} a^(i-j) (x_i.y_j) z_j + a^(i+1) x_i U_in
//   backward in time  out_i = sum_{j>=i} a^(j-i) (x_i.y_j) z_j + a^(n-1-i) x_i U_in
// and U_out = a^n U_in + sum_j u_j y_j z_j^T with u_j = a^(n-1-j) forward and
// a^(j+1) backward (n tokens).  The attention itself is (x,y,z) = (q,k,v)
// forward; its gradients are dq = (dout,v,k) forward, dk = (v,dout,q) and
// dv = (k,q,dout) backward in time.  Cut into segments, the walk needs only
// each segment's incoming state: a state pass forms every segment's own sum,
// a scan joins them, and the segments are walked side by side.
#pragma once

#include "lla_common.cuh"

namespace lla {

constexpr int kLinTile = 128;     // tokens per tile; segments are whole tiles
constexpr int kLinMaxSeg = 256;   // segments of one sequence, where it is not cut for kLinWalkTiles
// Tiles of one walk on the tensor cores.  Its state stays in one accumulator, which is not rounded to nearest: with
// a = 1 and terms of one sign it falls short by about 2.3e-6 a tile (measured).  256 tiles hold that to 6e-4, against
// the 2^-9 and more of the state operand's own rounding, and the next segment starts from a state of fp32 accuracy;
// whole walks of 4096 tiles were 2.8e-3 short, growing with T.  152 heads of 65536 tokens, D = 128, without a state:
// 1513 us whole, 2410 so (a pass over k and v for the states); up to 32768 tokens nothing is cut for it.
constexpr int kLinWalkTiles = 256;
constexpr int kLinMaxJobs = 3;

struct LinJob {
    const void *x, *y, *z;  // [BH][T][dx], [BH][T][dx], [BH][T][dz]; x unused by a state pass
    void *out;              // [BH][T][dz]
    const float *init;      // incoming states, nullptr: zero.  One per (bh, segment); a state pass has one only
                            // over whole sequences on the tensor cores, and adds it, decayed, to its sum
    long long init_bh, init_seg;  // strides in floats between heads and segments
    int init_t;             // the states in `init` are stored [dz][dx]
    float *final_;          // walk of one segment: U_out [BH][dx][dz], nullable; state pass: [BH][nseg][dx][dz]
    int rev;                // backward in time
    int dx, dz;
};

struct LinWalk {
    LinJob job[kLinMaxJobs];
    int njobs;
    const float *log_decay;  // [H]
    const int32_t *lens;     // [B], nullable
    int B, H, T, nseg, seg_tiles;
    lla_dtype dt;
    int32_t *device_error;
    void *stream;
    int withhold;            // test hook: the walk's scores and the state pass's products are not issued
};

// exp(ld * n) for n >= 0.  The product's rounding error is carried into the
// result (|ld n| can be large), and ld is held above -1e4, where every power
// but the zeroth is 0 in fp32 anyway, so that 0 * ld is 0 for any ld.  A NaN
// passes the comparison and every power of it is NaN.
__device__ __forceinline__ float decay_pow(float ld, int n)
{
    ld = ld < -1e4f ? -1e4f : ld;
    const float p = ld * (float)n;
    const float e = fmaf(ld, (float)n, -p);
    return expf(p) * (1.f + e);
}

// tokens of sequence b that count: lens[b] (T without lens), -1 if out of range
__device__ __forceinline__ int lin_length(const int32_t *lens, int b, int T)
{
    if (lens == nullptr) return T;
    const int n = lens[b];
    return (n >= 0 && n <= T) ? n : -1;
}

// CUDA cores: fp32
cudaError_t linattn_simt(const LinWalk &W, bool states_only);
// tensor cores: bf16
bool linattn_tc_supported(lla_dtype dt);
cudaError_t linattn_tc(const LinWalk &W, bool states_only, bool dependent);

struct LinFwdArgs {
    const void *q, *k, *v;
    const float *log_decay;
    const int32_t *lens;
    const float *state_in;
    void *out;
    float *state_out;
    int B, H, T, dk, dv;
    lla_dtype dt;
    bool after_padding;  // the kernel before this call's first is zero_padding's
    void *workspace;
    int32_t *device_error;
    void *stream;
};

struct LinBwdArgs {
    const void *q, *k, *v, *dout;
    const float *log_decay;
    const int32_t *lens;
    const float *state_in, *dstate_out;
    void *dq, *dkey, *dval;
    float *dstate_in;
    int B, H, T, dk, dv;
    lla_dtype dt;
    bool after_padding;  // the kernel before this call's first is zero_padding's
    void *workspace;
    int32_t *device_error;
    void *stream;
};

struct LinDecodeArgs {
    float *state;
    const void *q, *k, *v;
    const float *log_decay;
    const int32_t *slots;
    float *out;
    int pool, B, H, dk, dv;
    lla_dtype dt;
    int clear_skipped;
    int32_t *device_error;
    void *stream;
};

size_t linattn_fwd_workspace_bytes(int B, int H, int T, int dk, int dv, lla_dtype dt);
cudaError_t linattn_fwd(const LinFwdArgs &A);
size_t linattn_bwd_workspace_bytes(int B, int H, int T, int dk, int dv, lla_dtype dt);
cudaError_t linattn_bwd(const LinBwdArgs &A);
cudaError_t linattn_decode(const LinDecodeArgs &A);

}  // namespace lla
