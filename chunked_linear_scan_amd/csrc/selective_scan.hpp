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

#include <utility>

#include "selective.hpp"

namespace cls {

constexpr int kScanCh = 64;       // channels of a workgroup
constexpr int kScanMaxStates = 64;
constexpr int kScanMaxSegs = 64;
constexpr int64_t kScanMaxTokenStride = int64_t(1) << 26;  // a tile's rows stay within 32-bit offsets

// Tokens per tile, and between checkpoints: the backward pass holds a tile's
// states and decays in registers, and its partial sums in LDS.
constexpr int kScanTile = 8;
// waves of a workgroup at 4 states each, up to a power of two (at 24 states two of 8 have none)
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

// An element at a wave-uniform pointer and a lane's byte offset.  The empty
// statement keeps the offset a 32-bit register in the block that uses it, where
// the compiler can see that the access takes it as such; widened once and for
// all ahead of a loop, it would cost 64-bit address arithmetic at every access.
template <typename T>
__device__ __forceinline__ const T& at_bytes(const T* p, uint32_t bytes) {
    asm volatile("" : "+v"(bytes));
    return *reinterpret_cast<const T*>(reinterpret_cast<const char*>(p) + bytes);
}
template <typename T>
__device__ __forceinline__ T& at_bytes(T* p, uint32_t bytes) {
    asm volatile("" : "+v"(bytes));
    return *reinterpret_cast<T*>(reinterpret_cast<char*>(p) + bytes);
}

// Where a workgroup works.
struct ScanPlace {
    int64_t b;
    int g, seg, ch;
    bool on;              // the lane has a channel; one past its group computes the group's last, unseen
    int64_t first, stop;  // the segment's tokens
    int64_t last;         // the end of those that count
};

__device__ __forceinline__ ScanPlace scan_place(const ScanParams& p, int seg0 = 0) {
    ScanPlace a;
    const uint32_t blocks = uint32_t(p.bpg) * uint32_t(p.G);
    const uint32_t row = blockIdx.x / blocks, blk = blockIdx.x % blocks;
    a.g = int(blk / uint32_t(p.bpg));
    a.b = row % uint32_t(p.batch);
    a.seg = int(row / uint32_t(p.batch)) + seg0;
    const int c = int(blk % uint32_t(p.bpg)) * kScanCh + int(threadIdx.x & 63);
    a.on = c < p.cpg;
    a.ch = a.g * p.cpg + (a.on ? c : p.cpg - 1);
    const int end = seq_end(p.seqlens, a.b, p.L);
    a.first = int64_t(a.seg) * p.seg_len;
    a.stop = a.first + p.seg_len < p.L ? a.first + p.seg_len : p.L;
    a.last = a.stop < end ? a.stop : end;
    return a;
}

// The rows of B or C of a tile for one wave: lane l holds token (l / 4) % 8 and
// state n0 + l % 4, which is how a 4x4x1 matrix instruction takes the 4 rows of
// its A operand, block by block; see outer().
static_assert(kScanTile == 8 && kScanK == 4, "half a wave holds a tile");

template <typename E>
struct ScanRows {
    typedef typename E::raw raw;
    const raw* at;    // the tile to be loaded, the same for all lanes
    int stride, row;  // of a token; the lane's token
    uint32_t off;     // the lane's byte offset
    bool on;
    raw r;

    __device__ __forceinline__ ScanRows(const void* v, const ScanStride& s, int64_t b, int g, int64_t first, int n0, int N,
                                        int lane) {
        at = static_cast<const raw*>(v) + b * s.b + g * s.g + first * s.t;
        stride = int(s.t);
        row = (lane >> 2) & 7;
        const int n = n0 + (lane & 3);
        on = n < N;
        off = uint32_t(row * stride + (on ? n : 0)) * uint32_t(sizeof(raw));
    }
    // Loads the tile; rem: the last of its rows that may be read (below 0: before the tile).
    __device__ __forceinline__ void load(int rem) {
        if (rem >= kScanTile - 1) r = at_bytes(at, off);
        else r = *(&at_bytes(at, off) - int64_t(row > rem ? row - rem : 0) * stride);
    }
    __device__ __forceinline__ void step(int dir) { at += dir * kScanTile * int64_t(stride); }
    __device__ __forceinline__ float get() const { return on ? E::get(r) : 0.0f; }
};

// The same rows as operands of vector instructions: each row of 16 lanes of
// q[i] holds tokens 4 i to 4 i + 3, and the instruction that uses one of the
// values broadcasts it within the row as it reads it (a DPP operand).  Rows 0
// and 2 of a wave hold tokens 0 to 3, rows 1 and 3 tokens 4 to 7: swapping
// them between two copies gives both.
__device__ __forceinline__ void row_quads(float rows, float (&q)[2]) {
    const auto r = __builtin_amdgcn_permlane16_swap(as_uint(rows), as_uint(rows), false, false);
    q[0] = as_float(r[0]);
    q[1] = as_float(r[1]);
}

// rows: as ScanRows gives them.  c[k] + value(T, k) v for the wave's four states k, where v is the lane's own: the
// matrix instruction multiplies 16 blocks of 4 rows by 4 columns (the lanes), with the rows of block T in all blocks.
template <int T>
__device__ __forceinline__ f32x4 outer(float rows, float v, f32x4 c = f32x4{0.f, 0.f, 0.f, 0.f}) {
    return __builtin_amdgcn_mfma_f32_4x4x1f32(rows, v, c, 4, T, 0);
}

// sum_k value(T, k) v[k].  The compiler does not fold a DPP operand into a
// multiply-add, hence the instructions themselves, and it does not look into
// them for the waits that their operands need: two wait states between a vector
// instruction's write and a DPP operand, and five where v comes from a 4x4
// matrix instruction (MATRIX).  s_nop N waits N + 1.
template <int T, bool MATRIX = false>
__device__ __forceinline__ float dot(const float* rows, const float (&v)[4]) {
    constexpr int I = (T & 3) * 4;
    float y;
    asm("s_nop %10\n\t"
        "v_mul_f32_dpp %0, %1, %2 row_newbcast:%6 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %0, %1, %3 row_newbcast:%7 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %0, %1, %4 row_newbcast:%8 row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %0, %1, %5 row_newbcast:%9 row_mask:0xf bank_mask:0xf"
        : "=&v"(y)
        : "v"(rows[T >> 2]), "v"(v[0]), "v"(v[1]), "v"(v[2]), "v"(v[3]), "n"(I), "n"(I + 1), "n"(I + 2), "n"(I + 3),
          "n"(MATRIX ? 5 : 1));
    return y;
}

// Folds segment s's contribution into v: exp(A sum dt') v + its own, for the
// wave's states.  With decays above 1 the whole segment's decay may be infinite
// in fp32 over a state that is zero or tiny, where the product is neither.  So
// it is applied as three equal factors (A3: A log2(e) / 3) of 2^100 at most:
// past that any state but zero overflows as the product does, and a zero stays
// one.  Decays below 1 take the same way: a branch for the others cost the
// gradients of 4 x 2048 x 1536 x 16 bf16 1-2 %, this 0.5 %.
struct ScanFold {
    float sd, own[kScanK];
    __device__ __forceinline__ void load(const ScanParams& p, int s, int64_t b, int ch, int n0) {
        const int64_t sb = int64_t(s) * p.batch + b;
        sd = p.seg_dt[sb * p.ch + ch];
#pragma unroll
        for (int k = 0; k < kScanK; ++k) own[k] = n0 + k < p.N ? p.seg_h[(sb * p.N + n0 + k) * p.ch + ch] : 0.0f;
    }
    template <typename V>
    __device__ __forceinline__ void apply(const float (&A3)[kScanK], V& v) const {
#pragma unroll
        for (int k = 0; k < kScanK; ++k) {
            const float f = fexp2(fminf(A3[k] * sd, 100.0f)), x = v[k];
            v[k] = fmaf(f, f * (f * x), own[k]);
        }
    }
};

// Segments from, from + step, ... (n of them), four at a time so that their
// loads are in flight together (eight measured 5 % slower over a whole call:
// registers).
constexpr int kFoldAtOnce = 4;

template <typename V>
__device__ __forceinline__ void scan_fold(const ScanParams& p, int from, int step, int n, int64_t b, int ch, int n0,
                                          const float (&A2)[kScanK], V& v) {
    float A3[kScanK];
#pragma unroll
    for (int k = 0; k < kScanK; ++k) A3[k] = A2[k] * (1.0f / 3.0f);
    for (int i = 0; i < n; i += kFoldAtOnce) {
        ScanFold f[kFoldAtOnce];
#pragma unroll
        for (int j = 0; j < kFoldAtOnce; ++j)
            if (i + j < n) f[j].load(p, from + step * (i + j), b, ch, n0);
#pragma unroll
        for (int j = 0; j < kFoldAtOnce; ++j)
            if (i + j < n) f[j].apply(A3, v);
    }
}

// The segments that a sequence is cut into, and their length in tokens (a
// multiple of the tile).
struct ScanCut { int64_t nseg, seg_len; };

}  // namespace cls
