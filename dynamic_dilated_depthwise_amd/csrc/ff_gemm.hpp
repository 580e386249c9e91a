// ff_gemm.hpp -- the tiled matrix product of the feed-forward operators, forward and backward:
//
//   out[q][p] = sum over k of P(p, k) Q(q, k)
//
// p runs along the output's rows in memory, q over its rows.  Each operand lies in memory either
// with its contraction along its rows (kAlong: element [index][k]) or down its columns (kDown:
// element [k][index]), so one kernel serves
//   y = x W^T          P = W along,  Q = x along
//   grad_x = dz W      P = W down,   Q = dz along
//   grad_W = dz^T x    P = x down,   Q = dz down
//
// A step of the contraction is 128 bytes of it (64 bfloat16 or 32 float32).  A step's tile of an
// operand is TILE * 128 bytes of LDS in 16-byte chunks, placed by an exclusive or of the chunk's
// number with bits of its row, so that the fragment reads of a wave spread over the banks.  The tiles of
// two to four steps are held (see form_of): one is computed while the next ones arrive.
//   DIRECT   the chunks go straight from memory to LDS (no registers, nothing to wait for but the
//            step's end); needs 16-byte aligned rows and whole chunks.  Chunks outside the
//            operand are asked for past the buffer's end, which reads zero.
//   else     through registers, any alignment and any size, element by element at the ends.
// Rows and columns outside the operands are zero in LDS, so that nothing that is not finite in one
// row of x reaches another's output.
#pragma once

#include <type_traits>

#include "ff_curves.hpp"
#include "ff_launch.hpp"
#include "seq_common.hpp"

namespace ddpm {
namespace ff {

using namespace ddpm::seq;

typedef __attribute__((address_space(3))) void lds_void;

enum Side { kAlong, kDown };
enum Epi { kStore, kLinear, kGated, kWeight };

constexpr int kStepBytes = 128;
template <typename T> constexpr int kStep = kStepBytes / (int)sizeof(T);  // elements of a step

constexpr uint32_t kRecords = 0x7fffffe0u, kOutside = 0x7ffffff0u;  // of a buffer; an offset past it

// All but this wave's last N loads to LDS are there and its own LDS accesses done; then the workgroup.
template <int N> __device__ __forceinline__ void arrive_but() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" :: "n"(N) : "memory");
}
__device__ __forceinline__ void arrive_lds() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Between a wave's writes to LDS and other lanes' reads of them: the hardware keeps their order, the
// compiler only a lane's own.
__device__ __forceinline__ void wave_order() { asm volatile("" ::: "memory"); }

// 16 bytes a lane from `off` behind `p` (uniform; zeros from kRecords on) to LDS at `at` (uniform) + 16 lane.
// In assembly, because the compiler takes the builtin for a write to all of LDS and makes the fragment
// reads behind it wait for it (grad_x 930 -> 570 TFLOP/s with loads between them).  It has no result, so
// no register is held by a load in flight; arrive_but waits for it.  m0 is one of the
// registers that the compiler holds nothing in (it refuses them in a list of clobbered ones); a change of it
// needs one wait state.
__device__ __forceinline__ void load_to_lds(const void *p, uint32_t off, char *at) {
    const uint64_t a = (uint64_t)p;
    const u32x4 r = {(uint32_t)a, (uint32_t)(a >> 32) & 0xffffu, kRecords, 0x00020000u};
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
                 :: "v"(off), "s"(r), "s"((uint32_t)(uintptr_t)(lds_void *)at));
}

// The bits that a row's chunk numbers are placed by.  kAlong: eight rows read at one chunk.  kDown,
// bfloat16: the transposing reads take four rows of 32 bytes in each of two lane groups, eight rows
// 0..3 and 8..11 (or 16 more, 4 more); float32: rows 8 apart, 64 bytes of each.
template <typename T, Side S, int CH>
__device__ __forceinline__ int swizzle(int row) {
    if constexpr (S == kAlong) return row & 7;
    else if constexpr (!Elem<T>::is_bf16) return (row >> 3 & 3) << 2 & (CH - 1);
    else if constexpr (CH >= 16) return ((row & 3) | (row >> 3 & 1) << 2) << 1;
    else return ((row >> 1 & 1) | (row >> 3 & 1) << 1) << 1 & (CH - 1);
}

// One operand's tile: TILE indices from `first` of `extent`, contraction from k0.  The gated product's
// tile of P has 16 of the gate's rows, the same 16 of the other half, and so on.
template <typename T, Side S, int TILE, int THREADS, bool DIRECT, bool GATED>
struct Tile {
    static constexpr int kPer = kVec<T>, kCh = S == kAlong ? 8 : TILE / kPer;
    static constexpr int kCount = TILE * 8 / THREADS;
    static_assert(TILE * 8 % THREADS == 0, "whole rounds of chunks");
    typedef std::conditional_t<DIRECT, uint32_t, int64_t> Offset;  // direct_ok: within 2^31 bytes
    const T *p;
    int64_t ld;
    Offset off[kCount];  // of the chunks in a step's tile, in bytes
    u32x4 r[DIRECT ? 1 : kCount];
    int columns;  // kDown, through registers: of the tile that are there

    __device__ __forceinline__ static int row_of(int i, int tid) { return (i * THREADS + tid) / kCh; }
    __device__ __forceinline__ static int chunk_of(int i, int tid) {
        return (i * THREADS + tid) % kCh ^ swizzle<T, S, kCh>(row_of(i, tid));
    }
    // Rows (kAlong) that are not there: zeros, or through registers the last one's, which nobody takes
    // (extent: of the index; gated: columns of the result).
    __device__ __forceinline__ void start(const void *base, int64_t ld_, int64_t first, int64_t extent, int64_t k0, int tid) {
        ld = ld_;
        const int64_t from = GATED ? first >> 1 : first;
#pragma unroll
        for (int i = 0; i < kCount; ++i) {
            const int row = row_of(i, tid), c = chunk_of(i, tid);
            if constexpr (S == kAlong) {
                const int64_t at = GATED ? (row >> 5 << 4) + (row & 15) : row, last = extent - from - 1;
                const int64_t there = (at <= last ? at : last) + (GATED && row & 16 ? extent : 0);
                off[i] = DIRECT && at > last ? kOutside : (Offset)(there * ld * sizeof(T)) + c * 16;
            } else {
                off[i] = DIRECT && first + c * kPer >= extent ? kOutside : (Offset)(row * ld * sizeof(T)) + c * 16;
            }
        }
        p = (const T *)base + (S == kAlong ? from * ld + k0 : k0 * ld + from);
        columns = (int)(extent - from < TILE ? extent - from : TILE);
    }
    __device__ __forceinline__ int64_t step() const { return S == kAlong ? kStep<T> : kStep<T> * ld; }  // elements to the next one's
    // Round i of the chunks of the step, of which `left` elements of the contraction are there, straight to LDS.
    __device__ __forceinline__ void ask(int i, char *lds, int64_t left, int tid) const {
        Offset o = off[i];
        if (left < kStep<T>) {
            const bool on = S == kAlong ? chunk_of(i, tid) * kPer < left : row_of(i, tid) < left;
            o = on ? o : kOutside;
        }
        load_to_lds(p, o, lds + (i * THREADS + wave_of(tid) * kWave) * 16);
    }
    // The step's chunks into registers; put: from there into LDS.  Only the contraction's last step and
    // the last tile of a kDown operand's columns look at how many elements are there.
    __device__ __forceinline__ void fetch(int64_t left, int tid) {
        const bool whole = left >= kStep<T>;
#pragma unroll
        for (int i = 0; i < kCount; ++i) {
            const int row = row_of(i, tid), c = chunk_of(i, tid) * kPer;
            const char *at = (const char *)p + off[i];
            if constexpr (S == kAlong) {
                if (whole) r[i] = *(const u32x4_a2 *)at;
                else r[i] = load_vec<T>((const T *)at, left - c);
            } else {
                const bool on = whole || row < left;
                at -= on ? 0 : row * ld * (int64_t)sizeof(T);
                if (columns == TILE) r[i] = *(const u32x4_a2 *)at;
                else r[i] = load_vec<T>((const T *)at, columns - c);
                if (!on) r[i] = u32x4{0, 0, 0, 0};
            }
        }
    }
    __device__ __forceinline__ void put(char *lds, int tid) const {
#pragma unroll
        for (int i = 0; i < kCount; ++i) *(u32x4 *)(lds + (i * THREADS + tid) * 16) = r[i];
    }
};

// The bfloat16 next to a number: the largest for those above it, so that what it leaves of them is finite.
constexpr float kMostBf16 = 3.38953139e38f;
__device__ __forceinline__ float within_bf16(float v) { return __builtin_amdgcn_fmed3f(v, -kMostBf16, kMostBf16); }
__device__ __forceinline__ float first_term(float v) { return round_to_bf16(within_bf16(v)); }

// A float32 as three bfloat16 (8 + 8 + 8 bits, the float32 itself down to the subnormals).  Of the nine
// products of two such numbers the six above 2^-25 of the whole are taken, so that a float32 product
// costs six bfloat16 matrix instructions (96 cycles where the float32 ones take 256) at float32's
// precision.  The nearest bfloat16 is taken each time: with bits cut off instead, the terms left out
// would be four times larger and all of the product's sign.
constexpr int kParts = 3;
template <int N>
struct Terms {
    bf16x8 part[N];
};
typedef Terms<kParts> Split;
template <typename T> struct OperandOf { typedef Split type; };
template <> struct OperandOf<bf16_t> { typedef bf16x8 type; };
template <typename T> using Operand = typename OperandOf<T>::type;

// In pairs, as the conversion takes them: 13 instructions for two values.
__device__ __forceinline__ Split split_of(const f32x4 &a, const f32x4 &b) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    u32x4 part[kParts];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        f32x2 v = e < 2 ? f32x2{a[2 * e], a[2 * e + 1]} : f32x2{b[2 * e - 4], b[2 * e - 3]};
#pragma unroll
        for (int k = 0; k < kParts; ++k) {
            const f32x2 c = k == 0 ? f32x2{within_bf16(v[0]), within_bf16(v[1])} : v;
            const uint32_t t = __builtin_bit_cast(uint32_t, __builtin_convertvector(c, bf16x2_t));
            part[k][e] = t;
            v[0] -= __uint_as_float(t << 16);
            v[1] -= __uint_as_float(t & 0xffff0000u);
        }
    }
    Split r;
#pragma unroll
    for (int k = 0; k < kParts; ++k) r.part[k] = __builtin_bit_cast(bf16x8, part[k]);
    return r;
}

// acc[j] += p q[j], the smallest terms first; neighbouring instructions have different results.
template <int NQ>
__device__ __forceinline__ void multiply(f32x4 (&acc)[NQ], const bf16x8 &p, const bf16x8 (&q)[NQ]) {
#pragma unroll
    for (int j = 0; j < NQ; ++j) acc[j] = mma(p, q[j], acc[j]);
}
template <int NQ, int N>
__device__ __forceinline__ void multiply(f32x4 (&acc)[NQ], const bf16x8 &p, const Terms<N> (&q)[NQ]) {
#pragma unroll
    for (int k = N - 1; k >= 0; --k)
#pragma unroll
        for (int j = 0; j < NQ; ++j) acc[j] = mma(p, q[j].part[k], acc[j]);
}
template <int NQ>
__device__ __forceinline__ void multiply(f32x4 (&acc)[NQ], const Split &p, const Split (&q)[NQ]) {
#pragma unroll
    for (int order = kParts - 1; order >= 0; --order)
#pragma unroll
        for (int k = order; k >= 0; --k)
#pragma unroll
            for (int j = 0; j < NQ; ++j) acc[j] = mma(p.part[k], q[j].part[order - k], acc[j]);
}
__device__ __forceinline__ bf16x8 ones_frag() {
    bf16x8 f;
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = (__bf16)1.f;
    return f;
}
// sum[j] += the sums of q[j] over the contraction, in every row.
template <int NQ>
__device__ __forceinline__ void add_up(f32x4 (&sum)[NQ], const bf16x8 (&q)[NQ]) {
    multiply<NQ>(sum, ones_frag(), q);
}
template <int NQ, int N>
__device__ __forceinline__ void add_up(f32x4 (&sum)[NQ], const Terms<N> (&q)[NQ]) {
    multiply<NQ>(sum, ones_frag(), q);
}

// Fragments: slot e of lane group g stands for contraction index 8 g + e of a run of 32.
template <typename T, Side S, int TILE>
struct Reader {
    static constexpr int kCh = S == kAlong ? 8 : TILE / kVec<T>, kRow = kCh * 16;
    uint32_t base;
    __device__ __forceinline__ void start(int lane) {
        const int l16 = lane % 16, g = lane / 16;
        if constexpr (S == kAlong) {
            base = l16 * kRow + (((Elem<T>::is_bf16 ? g : 2 * g) ^ (l16 & 7)) << 4);
        } else if constexpr (Elem<T>::is_bf16) {
            const int k = 8 * g + l16 / 4;
            base = k * kRow + ((swizzle<T, S, kCh>(k) | (l16 % 4) / 2) << 4) + (l16 & 1) * 8;
        } else {
            const int k = 8 * g;
            base = k * kRow + ((swizzle<T, S, kCh>(k) | l16 / 4) << 4) + (l16 % 4) * 4;
        }
    }
    // Of the 16 indices from 16 * t, run s of the step.
    __device__ __forceinline__ Operand<T> get(const char *lds, int t, int s) const {
        if constexpr (S == kAlong && Elem<T>::is_bf16) {
            return *(const bf16x8 *)(lds + t * (16 * kRow) + (base ^ s * 64));
        } else if constexpr (S == kAlong) {
            return split_of(*(const f32x4 *)(lds + t * (16 * kRow) + base), *(const f32x4 *)(lds + t * (16 * kRow) + (base ^ 16)));
        } else if constexpr (Elem<T>::is_bf16) {
            typedef __attribute__((address_space(3))) s16x4 *lds_ptr;
            const char *at = lds + (base ^ t * 32) + s * (32 * kRow);
            const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)at);
            const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(at + 4 * kRow));
            u16x8 r;
#pragma unroll
            for (int e = 0; e < 4; ++e) { r[e] = (uint16_t)a[e]; r[4 + e] = (uint16_t)b[e]; }
            return __builtin_bit_cast(bf16x8, r);
        } else {
            f32x4 a, b;
            const char *at = lds + (base ^ t * 64);
#pragma unroll
            for (int e = 0; e < 4; ++e) { a[e] = *(const float *)(at + e * kRow); b[e] = *(const float *)(at + (4 + e) * kRow); }
            return split_of(a, b);
        }
    }
};

// Four neighbouring elements (element-aligned), widened.
template <typename T>
__device__ __forceinline__ f32x4 load_four(const T *p) {
    if constexpr (Elem<T>::is_bf16) {
        const u16x4 u = *(const u16x4_a2 *)p;
        return f32x4{bf16_bits_to_f32(u[0]), bf16_bits_to_f32(u[1]), bf16_bits_to_f32(u[2]), bf16_bits_to_f32(u[3])};
    } else {
        return *(const f32x4_a4 *)p;
    }
}

// Eight neighbouring elements: of a vector in memory (element-aligned), the first n of them.
template <typename T>
__device__ __forceinline__ void read8(const T *p, int64_t n, float (&v)[8]) {
    if constexpr (Elem<T>::is_bf16) {
        widen<T>(load_vec<T>(p, n), v);
    } else {
        float a[4], b[4];
        widen<T>(load_vec<T>(p, n), a);
        widen<T>(load_vec<T>(p + (n > 4 ? 4 : 0), n - 4), b);
#pragma unroll
        for (int e = 0; e < 4; ++e) { v[e] = a[e]; v[4 + e] = b[e]; }
    }
}
template <typename T>
__device__ __forceinline__ void write8(T *p, int64_t n, const float (&v)[8]) {
    if (n >= 8) {
        u32x4 w[sizeof(T) / 2];
        if constexpr (Elem<T>::is_bf16) {
#pragma unroll
            for (int e = 0; e < 4; ++e) w[0][e] = (uint32_t)f32_to_bf16_bits(v[2 * e]) | (uint32_t)f32_to_bf16_bits(v[2 * e + 1]) << 16;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e / 4][e % 4] = __float_as_uint(v[e]);
        }
#pragma unroll
        for (int h = 0; h < (int)sizeof(T) / 2; ++h) *(u32x4_a2 *)(p + h * kVec<T>) = w[h];
    } else {
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (e < n) p[e] = Elem<T>::from_f32(v[e]);
    }
}

// The bias of eight columns from p: of the gate's or the only half (half 0), or of the other (half 1).
template <typename T>
__device__ __forceinline__ void bias8(const Product &a, int64_t p, int half, float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.f;
    const int64_t at = half * a.np + p;
    if (p >= a.np) return;
    if (a.grad != nullptr) read8<float>(a.kept + at, a.np - p, v);
    else if (a.bias != nullptr) read8<T>((const T *)a.bias + at, a.np - p, v);
}
// For the backward, in float32.
__device__ __forceinline__ void keep8(const Product &a, int64_t p, int half, const float (&v)[8]) {
    if (a.kept != nullptr && a.grad == nullptr && p < a.np) write8<float>(a.kept + half * a.np + p, a.np - p, v);
}
// dz: rounded to bfloat16 alone it would make the gradients' error 1.4 times that of their own rounding, so
// that what the rounding leaves is kept beside it, `low` elements behind (0: the values are bfloat16's, or
// T is float32).  An infinity is the largest number and an infinity.
template <typename T>
__device__ __forceinline__ void write_dz(T *p, int64_t low, int64_t n, float (&v)[8]) {
    if constexpr (Elem<T>::is_bf16) {
        if (low != 0) {
            float rest[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float t = first_term(v[e]);
                rest[e] = v[e] - t;
                v[e] = t;
            }
            write8<T>(p + low, n, rest);
        }
    }
    write8<T>(p, n, v);
}
// Row q of dz: its zeros behind the last of `width` columns, up to a whole chunk.
template <typename T>
__device__ __forceinline__ void pad_row(T *row, int64_t low, int64_t width) {
    for (int64_t c = width; c % kVec<T> != 0; ++c) row[c] = row[low + c] = 0;
}
// dz of eight columns from p: grad act'(z); gated: grad u act'(g) and grad act(g).
template <typename T>
__device__ __forceinline__ void finish_dz(T *row, int64_t low, int64_t p, int64_t N, const T *grad, int act, const float (&z)[8]) {
    const int64_t n = N - p;
    float g[8], v[8], d[8];
    read8<T>(grad + p, n, g);
    slopes(z, v, d, act);
#pragma unroll
    for (int e = 0; e < 8; ++e) d[e] *= g[e];
    write_dz<T>(row + p, low, n, d);
    if (n <= 8) pad_row(row, low, N);
}
template <typename T>
__device__ __forceinline__ void finish_gated_dz(T *row, int64_t low, int64_t p, int64_t N, const T *grad, int act,
                                                const float (&z)[8], const float (&u)[8]) {
    const int64_t n = N - p;
    float g[8], v[8], d[8];
    read8<T>(grad + p, n, g);
    slopes(z, v, d, act);
#pragma unroll
    for (int e = 0; e < 8; ++e) { d[e] = g[e] * u[e] * d[e]; v[e] = g[e] * v[e]; }
    write_dz<T>(row + p, low, n, d);
    write_dz<T>(row + N + p, low, n, v);
    if (n <= 8) pad_row(row, low, 2 * N);
}

// What follows the product for eight neighbouring columns p of row q: z without its bias.
template <typename T>
__device__ __forceinline__ void finish_linear(const Product &a, int64_t q, int64_t p, float (&z)[8], const float (&bias)[8]) {
    const int64_t n = a.np - p;
    if (q >= a.nq || n <= 0) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] += bias[e];
    if (a.grad != nullptr) {
        finish_dz<T>((T *)a.out + q * padded(a.np, Elem<T>::is_bf16), a.low, p, a.np, (const T *)a.grad + q * a.grad_ld, a.act, z);
        return;
    }
    if (a.saved != nullptr) write8<float>(a.saved + q * a.np + p, n, z);
    activate(z, a.act);
    if (a.residual != nullptr) {
        float r[8];
        read8<T>((const T *)a.residual + q * a.residual_ld + p, n, r);
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] += r[e];
    }
    write8<T>((T *)a.out + q * a.np + p, n, z);
}
// Of the gated product: columns p of the gate's half and of the other's.
template <typename T>
__device__ __forceinline__ void finish_gated(const Product &a, int64_t q, int64_t p, float (&g)[8], float (&u)[8],
                                             const float (&gb)[8], const float (&ub)[8]) {
    const int64_t n = a.np - p;
    if (q >= a.nq || n <= 0) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) { g[e] += gb[e]; u[e] += ub[e]; }
    if (a.grad != nullptr) {
        finish_gated_dz<T>((T *)a.out + q * padded(2 * a.np, Elem<T>::is_bf16), a.low, p, a.np, (const T *)a.grad + q * a.grad_ld,
                           a.act, g, u);
        return;
    }
    if (a.saved != nullptr) {
        float *s = a.saved + q * 2 * a.np + p;
        write8<float>(s, n, g);
        write8<float>(s + a.np, n, u);
    }
    activate(g, a.act);
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] *= u[e];
    write8<T>((T *)a.out + q * a.np + p, n, g);
}

// WP * WQ waves of 16 MP by 16 NQ each.
template <typename T, Side SP, Side SQ, Epi E, int WP, int WQ, int MP, int NQ, int STAGES, bool DIRECT>
struct Gemm {
    static constexpr int kThreads = WP * WQ * kWave, kP = WP * MP * 16, kQ = WQ * NQ * 16;
    static constexpr int kStageBytes = (kP + kQ) * kStepBytes;
    static constexpr int kLd = 16 * MP + 4;  // floats of a row of the result in LDS
    static constexpr int kOutBytes = WP * WQ * 16 * kLd * 4;
    static constexpr int kStages = DIRECT ? STAGES : 2;
    static constexpr int kLds = kStages * kStageBytes > kOutBytes ? kStages * kStageBytes : kOutBytes;

    static constexpr int64_t kSlot = (int64_t)kP * kQ + (E == kWeight ? kQ : 0);  // floats of a piece's result

    // Where tile `id` starts: neighbours take eight tiles of q for each tile of p, so that both stay in the L2.
    __device__ __forceinline__ static void place(const Product &a, uint32_t id, int64_t &p0, int64_t &q0) {
        constexpr uint32_t kBand = 8;
        const uint32_t band = id / (kBand * a.tiles_p), in_band = id - band * kBand * a.tiles_p;
        const uint32_t rows = a.tiles_q - band * kBand < kBand ? a.tiles_q - band * kBand : kBand;
        q0 = (int64_t)(band * kBand + in_band % rows) * kQ;
        p0 = (int64_t)(in_band / rows) * kP;
    }

    __device__ static void run(const Product &a, char *lds) {
        const int tid = threadIdx.x, wave = wave_of(tid), lane = tid % kWave;
        const int wp = wave % WP, wq = wave / WP;
        // whole tiles first, then the pieces of the last ones, each kind in stretches of an XCD
        uint32_t tile, piece = 0, slot = 0;
        if (blockIdx.x < a.whole) {
            tile = xcd_contiguous((int)blockIdx.x, (int)a.whole);
        } else {
            slot = xcd_contiguous((int)(blockIdx.x - a.whole), (int)(gridDim.x - a.whole));
            const uint32_t cut = a.tiles_p * a.tiles_q - a.whole;
            piece = slot / cut;
            tile = a.whole + slot - piece * cut;
        }
        int64_t p0, q0;
        place(a, tile, p0, q0);
        const int64_t k0 = piece * a.run, k1 = blockIdx.x < a.whole || k0 + a.run > a.nk ? a.nk : k0 + a.run;
        float *part = blockIdx.x < a.whole ? nullptr : a.part + slot * kSlot;

        Tile<T, SP, kP, kThreads, DIRECT, E == kGated> tile_p;
        Tile<T, SQ, kQ, kThreads, DIRECT, false> tile_q;
        tile_p.start(a.p, a.p_ld, p0, a.np, k0, tid);
        tile_q.start(a.q, a.q_ld, q0, a.nq, k0, tid);
        Reader<T, SP, kP> read_p;
        Reader<T, SQ, kQ> read_q;
        read_p.start(lane);
        read_q.start(lane);

        f32x4 acc[MP][NQ], sum[E == kWeight ? NQ : 1];
#pragma unroll
        for (int i = 0; i < MP; ++i)
#pragma unroll
            for (int j = 0; j < NQ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < (E == kWeight ? NQ : 1); ++j) sum[j] = f32x4{0.f, 0.f, 0.f, 0.f};
        const bool sums = E == kWeight && p0 == 0 && wp == 0;

        // One step; between(n) is called before the n-th of its kBetween runs of matrix instructions.
        constexpr int kBetween = kStep<T> / 32 * MP;
        const auto compute = [&](const char *at, auto between) {
#pragma unroll
            for (int s = 0; s < kStep<T> / 32; ++s) {
                Operand<T> fq[NQ];
#pragma unroll
                for (int j = 0; j < NQ; ++j) fq[j] = read_q.get(at + kP * kStepBytes, wq * NQ + j, s);
                if constexpr (E == kWeight) {
                    if (sums) add_up<NQ>(sum, fq);
                }
#pragma unroll
                for (int i = 0; i < MP; ++i) {
                    between(s * MP + i);
                    multiply<NQ>(acc[i], read_p.get(at, wp * MP + i, s), fq);
                }
            }
            // The splits' vector instructions between the products: left in runs, they and the matrix
            // instructions do not overlap (39 % and 57 % of the cycles; 4096^3 597 -> 577 us,
            // 602 since the splits hold operands to bfloat16's range).
            if constexpr (!Elem<T>::is_bf16) {
                constexpr int kProducts = 6 * MP * NQ, kVector = 52 * (MP + NQ) / kProducts + 1;
#pragma unroll
                for (int n = 0; n < kProducts; ++n) {
                    __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
                    __builtin_amdgcn_sched_group_barrier(0x2, kVector, 0);
                }
            }
        };

        // With two terms of Q a step of the contraction is two: P's tile with that of Q's first term, then again
        // with the second one's (behind each other, so that the L2 has P's the second time).
        constexpr bool kMayTwo = Elem<T>::is_bf16 && (E == kStore || E == kWeight);
        const bool two = kMayTwo && a.low != 0;
        const int steps = (int)((k1 - k0 + kStep<T> - 1) / kStep<T>) << two;
        int64_t left = k1 - k0;
        bool second = false;
        const auto advance = [&] {
            if constexpr (kMayTwo) {
                second = two && !second;
                tile_p.p += second ? 0 : tile_p.step();
                tile_q.p += second ? a.low : tile_q.step() - a.low;
                left -= second ? 0 : kStep<T>;
            } else {
                tile_p.p += tile_p.step();
                tile_q.p += tile_q.step();
                left -= kStep<T>;
            }
        };
        if constexpr (DIRECT) {
            constexpr int kP1 = decltype(tile_p)::kCount, kAll = kP1 + decltype(tile_q)::kCount;
            const auto ask = [&](int i, char *at) {
                if (i < kP1) tile_p.ask(i, at, left, tid);
                else tile_q.ask(i - kP1, at + kP * kStepBytes, left, tid);
            };
            // Loads of kStages - 1 steps are under way behind the one that is computed; what is asked for
            // past the last step is nothing (zeros for LDS that nobody reads), so that a wave's count of
            // loads in flight is the same in every step.
#pragma unroll
            for (int t = 0; t < kStages - 1; ++t) {
#pragma unroll
                for (int i = 0; i < kAll; ++i) ask(i, lds + t * kStageBytes);
                advance();
            }
            int now = 0, next = kStages - 1;
            for (int s = 0; s < steps; ++s) {
                arrive_but<(kStages - 2) * kAll>();  // the step is there, and nobody reads the one before it any more
                // The chunks are asked for a few at a time: all of them at once would hold the wave up at
                // its first read (grad_x of 8192^3 bfloat16 1065 -> 867 us).
                compute(lds + now * kStageBytes, [&](int n) {
                    constexpr int kEach = (kAll + kBetween - 1) / kBetween;
#pragma unroll
                    for (int i = n * kEach; i < (n + 1) * kEach && i < kAll; ++i) ask(i, lds + next * kStageBytes);
                });
                advance();
                now = now + 1 == kStages ? 0 : now + 1;
                next = next + 1 == kStages ? 0 : next + 1;
            }
            arrive_but<0>();
        } else {
            tile_p.fetch(left, tid);
            tile_q.fetch(left, tid);
            for (int s = 0; s < steps; ++s) {
                char *now = lds + (s & 1) * kStageBytes;
                tile_p.put(now, tid);
                tile_q.put(now + kP * kStepBytes, tid);
                arrive_lds();
                if (s + 1 < steps) {
                    advance();
                    tile_p.fetch(left, tid);
                    tile_q.fetch(left, tid);
                }
                compute(now, [](int) {});
            }
            arrive_lds();
        }

        // Out through LDS, 16 rows of the wave's at a time, so that a lane has eight neighbouring columns
        // (the same ones in every row) and rows leave in whole runs.
        float *mine = (float *)lds + wave * 16 * kLd;
        constexpr bool kPair = E == kGated;
        constexpr int kPerRow = kPair ? MP : 2 * MP, kRows = kWave / kPerRow;  // lanes of a row, rows at a time
        const int c = lane % kPerRow, r0 = lane / kPerRow;
        const int at = kPair ? (c >> 1) * 32 + (c & 1) * 8 : c * 8;
        const int64_t p = kPair ? (p0 >> 1) + wp * MP * 8 + c * 8 : p0 + wp * MP * 16 + c * 8;
        float b0[8], b1[8];
        const bool keeps = q0 == 0 && piece == 0 && wq == 0 && r0 == 0;
        if constexpr (E == kLinear || E == kGated) {
            bias8<T>(a, p, 0, b0);
            if (keeps) keep8(a, p, 0, b0);
        }
        if constexpr (E == kGated) {
            bias8<T>(a, p, 1, b1);
            if (keeps) keep8(a, p, 1, b1);
        }
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
#pragma unroll
            for (int i = 0; i < MP; ++i) *(f32x4 *)(mine + (lane % 16) * kLd + 16 * i + 4 * (lane / 16)) = acc[i][j];
            wave_order();
            const int64_t q = q0 + (wq * NQ + j) * 16;
#pragma unroll 1
            for (int r = r0; r < 16; r += kRows) {
                float v[8], w[8];
                const f32x4 x0 = *(const f32x4 *)(mine + r * kLd + at), x1 = *(const f32x4 *)(mine + r * kLd + at + 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) { v[e] = x0[e]; v[4 + e] = x1[e]; }
                if constexpr (kPair) {
                    const f32x4 y0 = *(const f32x4 *)(mine + r * kLd + at + 16), y1 = *(const f32x4 *)(mine + r * kLd + at + 20);
#pragma unroll
                    for (int e = 0; e < 4; ++e) { w[e] = y0[e]; w[4 + e] = y1[e]; }
                }
                if (part != nullptr) {
                    float *t = part + ((wq * NQ + j) * 16 + r) * kP + wp * MP * 16 + at;
                    write8<float>(t, 8, v);
                    if constexpr (kPair) write8<float>(t + 16, 8, w);
                } else if constexpr (E == kLinear) {
                    finish_linear<T>(a, q + r, p, v, b0);
                } else if constexpr (E == kGated) {
                    finish_gated<T>(a, q + r, p, v, w, b0, b1);
                } else {
                    if (q + r < a.nq && p < a.np) write8<T>((T *)a.out + (q + r) * a.np + p, a.np - p, v);
                }
            }
            wave_order();
        }
        if constexpr (E == kWeight) {  // every row of `sum` holds the sums over k of Q
            if (sums && lane < 16) {
#pragma unroll
                for (int j = 0; j < NQ; ++j) {
                    const int at_q = (wq * NQ + j) * 16 + lane;
                    if (part != nullptr) part[kP * kQ + at_q] = sum[j][0];
                    else if (q0 + at_q < a.nq) ((T *)a.sums)[q0 + at_q] = Elem<T>::from_f32(sum[j][0]);
                }
            }
        }
    }

    // The sums of the pieces of the last tiles and what follows them.  A few lanes share the pieces of
    // eight neighbouring columns; their sums are joined in a fixed order.
    static constexpr int kFinishThreads = 256, kReds = E == kGated ? 17 : 9;
    static constexpr int kPerTile = (E == kGated ? kP / 2 : kP) * kQ / 8;
    static_assert(kPerTile % kFinishThreads == 0, "a workgroup stays in one tile");
    __device__ static void finish(const Product &a, float (*red)[kReds]) {
        constexpr int kCols = (E == kGated ? kP / 2 : kP) / 8;
        const int kLanes = finish_lanes(a.pieces), items = kFinishThreads / kLanes;
        const uint32_t cut = a.tiles_p * a.tiles_q - a.whole, blocks = kPerTile / items, tile = blockIdx.x / blocks;
        const int item = threadIdx.x % items, lane = threadIdx.x / items;
        const int i = (int)(blockIdx.x - tile * blocks) * items + item, row = i / kCols, c = i % kCols;
        const int at = E == kGated ? (c >> 1) * 32 + (c & 1) * 8 : c * 8;
        int64_t p0, q0;
        place(a, a.whole + tile, p0, q0);
        float v[8], w[8], sum = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = w[e] = 0.f;
        const bool sums = E == kWeight && p0 == 0 && c == 0;
        const float *t = a.part + ((int64_t)lane * cut + tile) * kSlot + row * kP + at;
        const int64_t far = (int64_t)kLanes * cut * kSlot;
#pragma unroll 4
        for (int s = lane; s < a.pieces; s += kLanes, t += far) {
            const f32x4 x0 = *(const f32x4 *)t, x1 = *(const f32x4 *)(t + 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) { v[e] += x0[e]; v[4 + e] += x1[e]; }
            if constexpr (E == kGated) {
                const f32x4 y0 = *(const f32x4 *)(t + 16), y1 = *(const f32x4 *)(t + 20);
#pragma unroll
                for (int e = 0; e < 4; ++e) { w[e] += y0[e]; w[4 + e] += y1[e]; }
            }
            if (E == kWeight && sums) sum += t[kP * kQ + row - (row * kP + at)];
        }
        if (kLanes > 1) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                red[threadIdx.x][e] = v[e];
                if constexpr (E == kGated) red[threadIdx.x][8 + e] = w[e];
            }
            if constexpr (E == kWeight) red[threadIdx.x][8] = sum;
            __syncthreads();
        }
        const int64_t q = q0 + row, p = E == kGated ? (p0 >> 1) + c * 8 : p0 + c * 8;
        if (lane == 0) {
            for (int l = 1; l < kLanes; ++l) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    v[e] += red[l * items + item][e];
                    if constexpr (E == kGated) w[e] += red[l * items + item][8 + e];
                }
                if constexpr (E == kWeight) sum += red[l * items + item][8];
            }
            if constexpr (E == kLinear) {
                float b[8];
                bias8<T>(a, p, 0, b);
                finish_linear<T>(a, q, p, v, b);
            } else if constexpr (E == kGated) {
                float g[8], u[8];
                bias8<T>(a, p, 0, g);
                bias8<T>(a, p, 1, u);
                finish_gated<T>(a, q, p, v, w, g, u);
            } else if (q < a.nq && p < a.np) {
                write8<T>((T *)a.out + q * a.np + p, a.np - p, v);
                if constexpr (E == kWeight) {
                    if (sums) ((T *)a.sums)[q] = Elem<T>::from_f32(sum);
                }
            }
        }
    }
};

template <typename G>
__global__ __launch_bounds__(G::kFinishThreads) void finish_kernel(const Product a) {
    __shared__ float red[G::kFinishThreads][G::kReds];
    G::finish(a, red);
}

template <typename G>
__global__ __launch_bounds__(G::kThreads, G::kThreads == 1024 ? 4 : 2) void gemm_kernel(const Product a) {
    __shared__ __attribute__((aligned(16))) char lds[G::kLds];
    G::run(a, lds);
}

}  // namespace ff
}  // namespace ddpm
