// What the forward and the backward pass of the selective scan share: the
// launch parameters, the cut of the work and the layout of checkpoints and
// workspaces.
//
// The work is cut into workgroups of 64 adjacent channels of one group and one
// segment of one sequence.  A lane is a channel; the states of a channel are
// dealt to the workgroup's NW waves, K to each.  So B and C are the same for
// all lanes of a wave, u and dt come in as rows of 64 adjacent channels, and
// the recurrence needs no exchange between lanes: only the sum over the states
// (y) crosses waves, through LDS, once per tile of tokens.
#pragma once

#include "selective.hpp"

namespace cls {

constexpr int kScanCh = 64;       // channels of a workgroup
constexpr int kScanMaxStates = 64;
constexpr int kScanMaxSegs = 64;

// Tokens per tile, and between checkpoints: the backward pass holds a tile's
// states and decays in registers, and its partial sums in LDS.
inline __host__ __device__ constexpr int scan_tile(int64_t N) { return N > 32 ? 8 : 16; }
// waves of a workgroup at 4 states each
inline __host__ __device__ constexpr int scan_waves(int64_t N) {
    return N <= 4 ? 1 : N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16;
}
constexpr int kScanK = 4;         // states of a wave

struct ScanStride { int64_t b, t, g; };

struct ScanParams {
    const void *u, *dt, *z, *B, *C;
    const float *A, *D, *dt_bias, *h0;
    const int32_t* seqlens;
    ScanStride su, sdt, sz, sB, sC;
    int batch, L, ch, N, G;
    int cpg;     // channels of a group
    int bpg;     // channel blocks of a group
    int nseg, seg_len;
    int softplus;
    // forward
    void* y;
    float* h_last;
    float* ckpt;    // [batch][tiles][N][ch]
    float* seg_h;   // [nseg][batch][N][ch]: a segment's state from zero
    float* seg_dt;  // [nseg][batch][ch]: a segment's summed steps
    // backward
    const void* dy;
    ScanStride sdy;
    const float* dh_last;
    void *du, *ddt, *dz, *dB, *dC;
    float *dA, *dD, *dbias, *dh0;
    float* part_bc;  // [blocks of the group][batch][L][G][2][N]: dB and dC of one channel block
    float* part_a;   // [batch * nseg][N + 2][ch]: dA, then dD, then ddt_bias
};

// The segments that a sequence is cut into, and their length in tokens (a
// multiple of the tile).
struct ScanCut { int64_t nseg, seg_len; };

}  // namespace cls
