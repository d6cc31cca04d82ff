// Linear attention with one decay per head: how a call is cut into segments,
// the scan that joins their states, and which kernels walk them.
#include "fwd_tc.cuh"
#include "launch.cuh"
#include "linattn.cuh"
#include "sm100.cuh"

namespace lla {
namespace {

struct Segments {
    int n, tiles;  // how many, tiles of each
};

int tiles_of(int T) { return T > 0 ? (int)(((long long)T + kLinTile - 1) / kLinTile) : 1; }

// What the kernels of a call are estimated to take, in microseconds, fitted to
// measured times: a CTA's start and end, a tile of 128 tokens, and for a state
// pass the scan of its states and the launches.  fp32: a tile's products on
// the CUDA cores (11 us at d = 32, 20 at 64, 44 at 128).  Lengths of a padded
// batch are not known here; its rows count as full.
struct Cost {
    int sms;
    double walk_start, walk_tile, sum_start, sum_tile, scan, launches;

    Cost(int dk, int dv, lla_dtype dt) : sms(sm_count())
    {
        if (!linattn_tc_supported(dt)) {
            walk_start = sum_start = 3.0;
            walk_tile = 6.0 + 0.00083 * (64.0 * dk + dv * (2.0 * dk + 64.0));
            sum_tile = 0.35 * walk_tile;
            launches = 5.0;
        } else if (dk > 64 || dv > 64) {
            walk_start = 5.0, walk_tile = 3.3, sum_start = 8.0, sum_tile = 2.1, launches = 3.3;
        } else {
            walk_start = 4.5, walk_tile = 2.5, sum_start = 5.0, sum_tile = 1.4, launches = 3.3;
        }
        scan = 0.04 * dk * dv / 16384;
    }
    double rounds(long long ctas) const { return (double)((ctas + sms - 1) / sms); }
    double walk(long long units, const Segments &c) const
    {
        return rounds(units * c.n) * (c.tiles * walk_tile + walk_start);
    }
    double sum(int tiles) const { return tiles * sum_tile + sum_start; }
    double states(long long units, const Segments &c) const
    {
        return rounds(units * c.n) * sum(c.tiles) + scan * (double)(units * c.n) + launches;
    }
    // one state pass over whole sequences that runs beside whole walks, on the SMs that those leave: a pass is
    // the shorter, so an SM that no walk takes does one or more
    double behind(long long walks, long long passes, int tiles) const
    {
        const Segments whole{1, tiles};
        const long long idle = (long long)rounds(walks) * sms - walks;
        const long long left = passes - idle * (long long)((tiles * walk_tile + walk_start) / sum(tiles));
        return walk(walks, whole) + launches + (left > 0 ? rounds(left) * sum(tiles) : 0.0);
    }
};

// How a call runs.  Its walks (`walks` of them, counted in heads) go over whole
// sequences, or in segments side by side whose incoming states `passes` state
// passes and the scan form first: the cheapest cut into at most kLinMaxSeg
// segments of whole tiles (more where bf16 walks of at most kLinWalkTiles need
// them).  A state that is handed out (`state`) comes with split walks from the
// scan.  Whole walks in fp32 hand it out themselves; those in bf16, whose own
// state is only as accurate as their output, leave it to one state pass behind
// them.
struct Plan {
    Segments cut;
    size_t part;  // bytes of one pass's states
    bool split() const { return cut.n > 1; }
};

Plan plan(int B, int H, int T, int dk, int dv, lla_dtype dt, int jobs, int passes, bool state)
{
    const long long BH = (long long)B * H, walks = jobs * BH;
    const int tiles = tiles_of(T);
    const Cost c(dk, dv, dt);
    const bool tc = linattn_tc_supported(dt);
    const int fewest = tc ? (tiles + kLinWalkTiles - 1) / kLinWalkTiles : 1;
    Segments best{1, tiles};
    double least = state && tc ? c.behind(walks, BH, tiles) : c.walk(walks, best);
    for (int n = fewest > 2 ? fewest : 2;
         n == fewest || (n <= kLinMaxSeg && n <= tiles && walks * (n - 1) < 4LL * c.sms); n++) {
        const Segments s{n, (tiles + n - 1) / n};
        if ((tiles + s.tiles - 1) / s.tiles != n) continue;  // never of the fewest
        const double cost = c.walk(walks, s) + c.states(passes * BH, s);
        if (cost < least || n == fewest) {
            least = cost;
            best = s;
        }
    }
    return {best, best.n > 1 ? align_up((size_t)BH * best.n * dk * dv * sizeof(float), 256) : 0};
}

size_t plan_bytes(int B, int H, int T, int dk, int dv, lla_dtype dt, int jobs, int passes)
{
    // enough with and without the state
    const size_t a = plan(B, H, T, dk, dv, dt, jobs, passes, false).part;
    const size_t b = plan(B, H, T, dk, dv, dt, jobs, passes, true).part;
    return passes * (a > b ? a : b);
}

struct ScanJob {
    float *seg;         // [BH][nseg][dx][dz]: a segment's own sum on entry, its incoming state on return
    const float *init;  // [BH][dx][dz] or transposed, nullptr: zero
    float *final_;      // [BH][dx][dz], nullable; may be `init` itself when that is not transposed
    int init_t, rev;
};

struct Scan {
    ScanJob job[2];
    const float *log_decay;
    const int32_t *lens;
    int dx[2], dz[2];
    int H, T, nseg, seg_tiles;
    int32_t *device_error;
};

// incoming state of segment s+1 = a^(tokens of s) incoming(s) + sum(s), along
// the walk's direction.  A thread has four neighbouring elements of the state;
// the segments' sums are read kAhead at a time, the next batch before the last
// one is written, so that a long row of segments is not a row of round trips.
constexpr int kScanThreads = 128, kAhead = 8;

__global__ void __launch_bounds__(kScanThreads)
linattn_scan_kernel(const __grid_constant__ Scan S)
{
    const ScanJob &J = S.job[blockIdx.z];
    const int dx = S.dx[blockIdx.z], dz = S.dz[blockIdx.z], n = dx * dz;
    const int bh = blockIdx.y, b = bh / S.H;
    const int e = (blockIdx.x * kScanThreads + threadIdx.x) * 4;
    if (e >= n) return;
    sm100::grid_launch_dependents();
    const int len = lin_length(S.lens, b, S.T);
    if (len < 0) {
        sm100::grid_dependency_wait();  // what comes after this kernel counts on the one before it too
        if (e == 0 && S.device_error != nullptr) atomicCAS(S.device_error, 0, LLA_DEVERR_BAD_LENGTH);
        return;
    }
    const float ld = S.log_decay[bh % S.H];
    const long long seg_tok = (long long)S.seg_tiles * kLinTile;
    const float full = decay_pow(ld, (int)(seg_tok < S.T ? seg_tok : S.T));
    float4 run = make_float4(0.f, 0.f, 0.f, 0.f);
    if (J.init != nullptr) {
        const float *in = J.init + (long long)bh * n;
        if (J.init_t) {
            const float *at = in + (e % dz) * dx + e / dz;
            run = make_float4(at[0], at[dx], at[2 * dx], at[3 * dx]);
        } else {
            run = *reinterpret_cast<const float4 *>(in + e);
        }
    }
    float *seg = J.seg + (long long)bh * S.nseg * n + e;
    auto at = [&](int k) {  // the k-th segment of the walk
        return reinterpret_cast<float4 *>(seg + (long long)(J.rev ? S.nseg - 1 - k : k) * n);
    };
    sm100::grid_dependency_wait();  // the sums are the kernel's before this one
    float4 own[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; u++)
        if (u < S.nseg) own[u] = *at(u);
    for (int k0 = 0; k0 < S.nseg; k0 += kAhead) {
        float4 next[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; u++)
            if (k0 + kAhead + u < S.nseg) next[u] = *at(k0 + kAhead + u);
#pragma unroll
        for (int u = 0; u < kAhead; u++) {
            if (k0 + u >= S.nseg) break;
            const long long left = len - (long long)(J.rev ? S.nseg - 1 - (k0 + u) : k0 + u) * seg_tok;
            const float w = left >= seg_tok ? full : (left <= 0 ? 1.f : decay_pow(ld, (int)left));
            *at(k0 + u) = run;
            run.x = fmaf(w, run.x, own[u].x);
            run.y = fmaf(w, run.y, own[u].y);
            run.z = fmaf(w, run.z, own[u].z);
            run.w = fmaf(w, run.w, own[u].w);
        }
#pragma unroll
        for (int u = 0; u < kAhead; u++) own[u] = next[u];
    }
    if (J.final_ != nullptr) *reinterpret_cast<float4 *>(J.final_ + (long long)bh * n + e) = run;
}

// dependent: right behind the state pass whose sums it joins
cudaError_t run_scan(const Scan &S, int jobs, int BH, void *stream, bool dependent)
{
    int n = 0;
    for (int j = 0; j < jobs; j++) n = S.dx[j] * S.dz[j] > n ? S.dx[j] * S.dz[j] : n;
    const int per = 4 * kScanThreads;
    return launch_kernel(linattn_scan_kernel, dim3((unsigned)((n + per - 1) / per), (unsigned)BH, (unsigned)jobs),
                         kScanThreads, 0, stream, dependent, S);
}

// what the walks and the scan of one call share
template <typename Args>
void call_args(const Args &A, const Segments &c, LinWalk &W, Scan &S)
{
    W.log_decay = A.log_decay; W.lens = A.lens; W.B = A.B; W.H = A.H; W.T = A.T; W.dt = A.dt;
    W.nseg = c.n; W.seg_tiles = c.tiles; W.device_error = A.device_error; W.stream = A.stream;
    W.withhold = withhold_first_product() ? 1 : 0;
    S.log_decay = A.log_decay; S.lens = A.lens; S.H = A.H; S.T = A.T; S.nseg = c.n; S.seg_tiles = c.tiles;
    S.device_error = A.device_error;
}

LinJob job(const void *x, const void *y, const void *z, void *out, int dx, int dz, int rev)
{
    LinJob J{};
    J.x = x; J.y = y; J.z = z; J.out = out; J.dx = dx; J.dz = dz; J.rev = rev;
    return J;
}

void take_state(LinJob &J, const float *states, int nseg, int n, int transposed)
{
    J.init = states;
    J.init_bh = (long long)nseg * n;
    J.init_seg = n;
    J.init_t = transposed;
}

// dependent: right behind the scan whose states the walks take, behind the walks beside which a state pass runs,
// or behind the fill of the outputs' padding
cudaError_t walk(const LinWalk &W, bool states_only, bool dependent)
{
    return linattn_tc_supported(W.dt) ? linattn_tc(W, states_only, dependent) : linattn_simt(W, states_only);
}

// Whole walks, and behind those in bf16 the pass that forms the state they hand out: job `j` of W from `init`.
cudaError_t whole_walks(LinWalk W, int j, const float *init, float *state, bool dependent)
{
    const bool tc = linattn_tc_supported(W.dt);
    if (!tc) W.job[j].final_ = state;
    const cudaError_t e = walk(W, false, dependent);
    if (e != cudaSuccess || state == nullptr || !tc) return e;
    W.job[0] = W.job[j];
    W.njobs = 1;
    take_state(W.job[0], init, 1, W.job[0].dx * W.job[0].dz, 0);
    W.job[0].final_ = state;
    return walk(W, true, true);
}

}  // namespace

size_t linattn_fwd_workspace_bytes(int B, int H, int T, int dk, int dv, lla_dtype dt)
{
    return plan_bytes(B, H, T, dk, dv, dt, 1, 1);
}

cudaError_t linattn_fwd(const LinFwdArgs &A)
{
    const int BH = A.B * A.H, n = A.dk * A.dv;
    const Plan p = plan(A.B, A.H, A.T, A.dk, A.dv, A.dt, 1, 1, A.state_out != nullptr);
    LinWalk W{};
    Scan S{};
    call_args(A, p.cut, W, S);
    S.dx[0] = A.dk; S.dz[0] = A.dv;
    S.job[0].init = A.state_in; S.job[0].final_ = A.state_out;
    if (A.T == 0) {  // no tokens: the state is handed through
        S.nseg = 0;
        return A.state_out != nullptr ? run_scan(S, 1, BH, A.stream, false) : cudaSuccess;
    }
    W.job[0] = job(A.q, A.k, A.v, A.out, A.dk, A.dv, 0);
    W.njobs = 1;
    if (!p.split()) {
        take_state(W.job[0], A.state_in, 1, n, 0);
        return whole_walks(W, 0, A.state_in, A.state_out, A.after_padding);
    }
    float *seg = (float *)A.workspace;
    W.job[0].final_ = S.job[0].seg = seg;
    cudaError_t e = walk(W, true, A.after_padding);
    if (e == cudaSuccess) e = run_scan(S, 1, BH, A.stream, true);
    W.job[0].final_ = nullptr;
    take_state(W.job[0], seg, p.cut.n, n, 0);
    return e == cudaSuccess ? walk(W, false, true) : e;
}

size_t linattn_bwd_workspace_bytes(int B, int H, int T, int dk, int dv, lla_dtype dt)
{
    return plan_bytes(B, H, T, dk, dv, dt, 3, 2);
}

// dq walks (dout, v, k) forward in time on the transposed states S^T; dk and dv
// walk (v, dout, q) and (k, q, dout) backward on dS^T and dS, the gradients of
// the states.
cudaError_t linattn_bwd(const LinBwdArgs &A)
{
    const int BH = A.B * A.H, n = A.dk * A.dv;
    const Plan p = plan(A.B, A.H, A.T, A.dk, A.dv, A.dt, 3, 2, A.dstate_in != nullptr);
    LinWalk W{};
    Scan S{};
    call_args(A, p.cut, W, S);
    // job 0: dS [dk][dv] backward from dstate_out; job 1: S^T [dv][dk] forward from state_in
    S.dx[0] = A.dk; S.dz[0] = A.dv;
    S.job[0].init = A.dstate_out; S.job[0].final_ = A.dstate_in; S.job[0].rev = 1;
    S.dx[1] = A.dv; S.dz[1] = A.dk;
    S.job[1].init = A.state_in; S.job[1].init_t = 1;
    if (A.T == 0) {
        S.nseg = 0;
        return A.dstate_in != nullptr ? run_scan(S, 1, BH, A.stream, false) : cudaSuccess;
    }
    const LinJob dq = job(A.dout, A.v, A.k, A.dq, A.dv, A.dk, 0);
    const LinJob dkey = job(A.v, A.dout, A.q, A.dkey, A.dv, A.dk, 1);
    const LinJob dval = job(A.k, A.q, A.dout, A.dval, A.dk, A.dv, 1);
    const float *s0 = A.dstate_out, *s1 = A.state_in;
    if (p.split()) {
        float *ds = (float *)A.workspace, *st = (float *)((char *)A.workspace + p.part);
        W.njobs = 2;
        W.job[0] = dval;
        W.job[0].final_ = S.job[0].seg = ds;
        W.job[1] = dq;
        W.job[1].final_ = S.job[1].seg = st;
        cudaError_t e = walk(W, true, A.after_padding);
        if (e == cudaSuccess) e = run_scan(S, 2, BH, A.stream, true);
        if (e != cudaSuccess) return e;
        s0 = ds;
        s1 = st;
    }
    W.njobs = 3;
    W.job[0] = dq;
    W.job[1] = dkey;
    W.job[2] = dval;
    take_state(W.job[0], s1, p.cut.n, n, p.split() ? 0 : 1);
    take_state(W.job[1], s0, p.cut.n, n, 1);
    take_state(W.job[2], s0, p.cut.n, n, 0);
    return p.split() ? walk(W, false, true)
                     : whole_walks(W, 2, A.dstate_out, A.dstate_in, A.after_padding);
}

}  // namespace lla
