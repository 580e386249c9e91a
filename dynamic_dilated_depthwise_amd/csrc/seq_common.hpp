// seq_common.hpp -- device helpers of the sequence operators (layer norm, short causal
// convolution, selective scan): loads of any alignment, matrix fragments of either type.
//
// Fragments.  Every product runs in steps of 32 along its contraction.  A lane (l16 =
// lane % 16, g = lane / 16) holds eight elements of one row (A) or column (B) l16; slot
// e of group g stands for the contraction index
//     k(g, e) = 4g + e          (e < 4)
//               16 + 4g + e - 4 (e >= 4)
// Any assignment is right as long as A and B share it.  This one is what the accumulator
// layout gives (component v of group g is row 4g + v of a 16 x 16 tile), so two result
// tiles one above the other are the operand of the next product with no exchange between
// lanes, and what the transposing LDS read gives (four rows of a column per lane).  For
// float32 the same eight slots feed eight 16x16x4 products.
#pragma once

#include "common.hpp"

namespace ddpm {
namespace seq {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint16_t u16x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// Elements of one 16-byte vector.
template <typename T> constexpr int kVec = 16 / (int)sizeof(T);

// 16 bytes from `p`, which need only be aligned to its element, when n >= kVec of them
// are there; otherwise the n that are, and zeros.  Nothing past p[n - 1] is read.
template <typename T>
__device__ __forceinline__ u32x4 load_vec(const T *__restrict__ p, int64_t n) {
    u32x4 r = {0, 0, 0, 0};
    if (n >= kVec<T>) {
        r = *(const u32x4_a2 *)p;
    } else if (n > 0) {
        if constexpr (Elem<T>::is_bf16) {
            for (int e = 0; e < 7; ++e)
                if (e < n) r[e / 2] |= (uint32_t)p[e] << (16 * (e % 2));
        } else {
            for (int e = 0; e < 3; ++e)
                if (e < n) r[e] = __float_as_uint(p[e]);
        }
    }
    return r;
}

template <typename T>
__device__ __forceinline__ void widen(const u32x4 &r, float (&v)[kVec<T>]) {
    if constexpr (Elem<T>::is_bf16) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] = __uint_as_float(r[e] << 16);
            v[2 * e + 1] = __uint_as_float(r[e] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(r[e]);
    }
}

// V neighbouring elements of a row of `size`, as they lie in memory.  How they are reached:
//   kWhole  size is a multiple of V: a vector is there or not
//   kOdd    size is at least V: the last vector is read ending with the row and moved down
//   kShort  the row is shorter than a vector: element by element
// Every form reads only the row's own elements.
enum Reach { kWhole, kOdd, kShort };
inline Reach reach_of(int64_t size, int V) { return size % V == 0 ? kWhole : size > V ? kOdd : kShort; }

template <typename T, int V>
struct Raw {
    static constexpr int kWords = V * (int)sizeof(T) / 4, kPer = 4 / (int)sizeof(T);
    typedef uint32_t words __attribute__((ext_vector_type(kWords)));
    typedef uint32_t words_a __attribute__((ext_vector_type(kWords), aligned(2)));
    words r;
    // Elements c .. c + V - 1 of `row`, zeros past its end or (on = false) altogether; `row`
    // is readable in any case.
    template <Reach R>
    __device__ __forceinline__ void load(const T *__restrict__ row, int c, int size, bool on) {
        if constexpr (R == kWhole) {
            on = on && c < size;
            r = *(const words_a *)(row + (on ? c : 0));
            r = on ? r : words(0);
        } else if constexpr (R == kOdd) {
            on = on && c < size;
            const int over = on ? (c + V > size ? c + V - size : 0) : 0;
            r = *(const words_a *)(row + (on ? c - over : 0));
            r = on ? r : words(0);
            if (over > 0) {
                if constexpr (kPer == 2) {
                    if (over & 1) {
#pragma unroll
                        for (int k = 0; k < kWords; ++k) r[k] = r[k] >> 16 | (k + 1 < kWords ? r[k + 1] << 16 : 0);
                    }
                }
#pragma unroll
                for (int m = 1; m < kWords; m *= 2) {
                    if (over / kPer & m) {
#pragma unroll
                        for (int k = 0; k < kWords; ++k) r[k] = k + m < kWords ? r[k + m] : 0;
                    }
                }
            }
        } else {
            r = words(0);
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (on && c + e < size) {
                    if constexpr (kPer == 2) r[e / 2] |= (uint32_t)row[c + e] << (16 * (e % 2));
                    else r[e] = __float_as_uint(row[c + e]);
                }
        }
    }
    __device__ __forceinline__ float operator[](int e) const {
        if constexpr (kPer == 2) return __uint_as_float(e % 2 ? r[e / 2] & 0xffff0000u : r[e / 2] << 16);
        else return __uint_as_float(r[e]);
    }
    __device__ __forceinline__ void set(const float (&v)[V]) {
#pragma unroll
        for (int k = 0; k < kWords; ++k) {
            if constexpr (kPer == 2)
                r[k] = (uint32_t)f32_to_bf16_bits(v[2 * k]) | (uint32_t)f32_to_bf16_bits(v[2 * k + 1]) << 16;
            else
                r[k] = __float_as_uint(v[k]);
        }
    }
    // Into elements c .. of `row`, those before its end.
    template <Reach R>
    __device__ __forceinline__ void store(T *__restrict__ row, int c, int size) const {
        if (R == kWhole || c + V <= size) {
            if (c < size) *(words_a *)(row + c) = r;
            return;
        }
        words t = r;
        int left = size - c;
        T *p = row + c;
#pragma unroll
        for (int m = kWords / 2; m > 0; m /= 2) {  // halves, quarters: few stores for any length
            if (left >= m * kPer) {
#pragma unroll
                for (int k = 0; k < m; ++k) store_word(p + k * kPer, t[k]);
#pragma unroll
                for (int k = 0; k < kWords; ++k) t[k] = k + m < kWords ? t[k + m] : 0;
                p += m * kPer;
                left -= m * kPer;
            }
        }
        if (kPer == 2 && left > 0) *p = (T)(t[0] & 0xffffu);
    }
    __device__ static __forceinline__ void store_word(T *p, uint32_t w) {
        typedef uint32_t word_a __attribute__((aligned(2)));
        *(word_a *)p = w;
    }
};

// Four elements at `p` (element-aligned), the first n of them.
template <typename T>
__device__ __forceinline__ void store4(T *__restrict__ p, const f32x4 &v, int n) {
    if (n >= 4) {
        if constexpr (Elem<T>::is_bf16) {
            u16x4 u;
#pragma unroll
            for (int e = 0; e < 4; ++e) u[e] = f32_to_bf16_bits(v[e]);
            *(u16x4_a2 *)p = u;
        } else {
            *(f32x4_a4 *)p = v;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (e < n) p[e] = Elem<T>::from_f32(v[e]);
    }
}

__device__ __forceinline__ f32x4 load4(const float *__restrict__ p, int n) {
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    if (n >= 4) {
        v = *(const f32x4_a4 *)p;
    } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (e < n) v[e] = p[e];
    }
    return v;
}

// Workgroups go to the eight XCDs in turn; numbered like this, 32 neighbours at a time are on one,
// and what they share in its L2.  No more than 32, so that sequences of different lengths still
// spread over all XCDs.
__device__ __forceinline__ int64_t block_in_stretch() {
    constexpr int64_t kRow = 32, kAll = 8 * kRow;
    const int64_t id = blockIdx.x, first = id / kAll * kAll, at = id - first;
    return first + kAll <= gridDim.x ? first + at % 8 * kRow + at / 8 : id;
}

// The wave's number in its workgroup, as a scalar: branches on it are then branches and not
// masks (left in a vector register it costs the scan's kernels a factor of two and more).
__device__ __forceinline__ int wave_of(int tid) { return __builtin_amdgcn_readfirstlane(tid / kWave); }

// The same number, which the compiler takes for a new one: addresses made from it inside a
// loop are made there and hold no registers between its turns.
__device__ __forceinline__ int afresh(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

// softplus in the form that neither overflows nor cancels.
__device__ __forceinline__ float softplus(float v) { return fmaxf(v, 0.f) + log1pf(expf(-fabsf(v))); }

// ------------------------------------------------------------------------------ fragments
struct FragF {
    float v[8];
};
template <typename T> struct FragOf { typedef FragF type; };
template <> struct FragOf<bf16_t> { typedef bf16x8 type; };
template <typename T> using Frag = typename FragOf<T>::type;

// LDS rows carry 16 bytes of padding, so that 16 rows read at one column start in different banks;
// bfloat16 rows of up to 64 columns 32, with which the transposing reads (four rows a lane group)
// spread as well (bank conflicts of the scan's backward 39 % -> 16 % of its LDS cycles).
template <typename T> constexpr int ld_of(int cols) { return cols + (Elem<T>::is_bf16 && cols <= 64 ? 16 : kVec<T>); }

__device__ __forceinline__ f32x4 mma(const bf16x8 &a, const bf16x8 &b, f32x4 c) { return mfma_16x16x32_bf16(a, b, c); }
// Two chains of four, so that fewer roundings follow each other (and the second starts at once).
__device__ __forceinline__ f32x4 mma(const FragF &a, const FragF &b, f32x4 c) {
    f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        c = mfma_16x16x4_f32(a.v[e], b.v[e], c);
        d = mfma_16x16x4_f32(a.v[e + 1], b.v[e + 1], d);
    }
    return c + d;
}

// Contraction along a row: `row` points at element k0 of the lane's own row.  near_frag is
// for products whose operands both run along rows: slot e of group g then stands for 8g + e,
// one 16-byte read (the two halves of row_frag, which matches col_frag, are fused by the
// compiler into a read with a short offset, at the price of an address register a tile).
__device__ __forceinline__ bf16x8 near_frag(const bf16_t *row, int g) { return *(const bf16x8 *)(row + 8 * g); }
__device__ __forceinline__ FragF near_frag(const float *row, int g) {
    const f32x4 a = *(const f32x4 *)(row + 8 * g), b = *(const f32x4 *)(row + 8 * g + 4);
    FragF r;
#pragma unroll
    for (int e = 0; e < 4; ++e) { r.v[e] = a[e]; r.v[4 + e] = b[e]; }
    return r;
}
__device__ __forceinline__ bf16x8 row_frag(const bf16_t *row, int g) {
    const u16x4 a = *(const u16x4 *)(row + 4 * g), b = *(const u16x4 *)(row + 16 + 4 * g);
    u16x8 r;
#pragma unroll
    for (int e = 0; e < 4; ++e) { r[e] = a[e]; r[4 + e] = b[e]; }
    return __builtin_bit_cast(bf16x8, r);
}
__device__ __forceinline__ FragF row_frag(const float *row, int g) {
    const f32x4 a = *(const f32x4 *)(row + 4 * g), b = *(const f32x4 *)(row + 16 + 4 * g);
    FragF r;
#pragma unroll
    for (int e = 0; e < 4; ++e) { r.v[e] = a[e]; r.v[4 + e] = b[e]; }
    return r;
}

// Contraction down the rows r0 .. r0 + 31 of an LDS tile, column c0 + l16.
__device__ __forceinline__ bf16x8 col_frag(const bf16_t *tile, int ld, int r0, int c0, int l16, int g) {
    typedef __attribute__((address_space(3))) s16x4 *lds_ptr;
    const bf16_t *p = tile + (r0 + 4 * g + l16 / 4) * ld + c0 + 4 * (l16 % 4);
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)p);
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + 16 * ld));
    u16x8 r;
#pragma unroll
    for (int e = 0; e < 4; ++e) { r[e] = (uint16_t)a[e]; r[4 + e] = (uint16_t)b[e]; }
    return __builtin_bit_cast(bf16x8, r);
}
__device__ __forceinline__ FragF col_frag(const float *tile, int ld, int r0, int c0, int l16, int g) {
    const float *p = tile + (r0 + 4 * g) * ld + c0 + l16;
    FragF r;
#pragma unroll
    for (int e = 0; e < 4; ++e) { r.v[e] = p[e * ld]; r.v[4 + e] = p[(16 + e) * ld]; }
    return r;
}

// Two result tiles, rows 0..15 and 16..31 of the contraction, as an operand; bf16 rounds.
template <typename T>
__device__ __forceinline__ Frag<T> pack_frag(const f32x4 &a, const f32x4 &b) {
    Frag<T> r;
    if constexpr (Elem<T>::is_bf16) {
#pragma unroll
        for (int e = 0; e < 4; ++e) { r[e] = (__bf16)a[e]; r[4 + e] = (__bf16)b[e]; }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) { r.v[e] = a[e]; r.v[4 + e] = b[e]; }
    }
    return r;
}

// A float32 as the sum of three bfloat16: 8 + 8 + 8 significant bits, so the sum is the
// float32 itself (down to the subnormals) and a product with a bfloat16 operand keeps
// float32's precision at three matrix instructions.
__device__ __forceinline__ void split3(float f, __bf16 &hi, __bf16 &mid, __bf16 &lo) {
    hi = (__bf16)f;
    const float r = f - (float)hi;
    mid = (__bf16)r;
    lo = (__bf16)(r - (float)mid);
}

// pack_frag in two bfloat16 terms, the second into `lo` (17 bits in all); float32 needs no second.
template <typename T>
__device__ __forceinline__ Frag<T> pack_frag2(const f32x4 &a, const f32x4 &b, Frag<T> &lo) {
    const Frag<T> hi = pack_frag<T>(a, b);
    if constexpr (Elem<T>::is_bf16) {
        f32x4 ra, rb;
#pragma unroll
        for (int e = 0; e < 4; ++e) { ra[e] = a[e] - (float)hi[e]; rb[e] = b[e] - (float)hi[4 + e]; }
        lo = pack_frag<T>(ra, rb);
    }
    return hi;
}
__device__ __forceinline__ f32x4 mma2(const bf16x8 &a, const bf16x8 &hi, const bf16x8 &lo, f32x4 c) {
    return mma(a, lo, mma(a, hi, c));
}
__device__ __forceinline__ f32x4 mma2(const FragF &a, const FragF &hi, const FragF &, f32x4 c) { return mma(a, hi, c); }

// Terms an exact float32 operand takes in the type's matrix products.
template <typename T> constexpr int kTerms = Elem<T>::is_bf16 ? 3 : 1;

// Four neighbouring elements of an LDS row, 4-element aligned.
__device__ __forceinline__ f32x4 lds4(const float *p) { return *(const f32x4 *)p; }
__device__ __forceinline__ f32x4 lds4(const bf16_t *p) {
    const u16x4 u = *(const u16x4 *)p;
    return f32x4{bf16_bits_to_f32(u[0]), bf16_bits_to_f32(u[1]), bf16_bits_to_f32(u[2]), bf16_bits_to_f32(u[3])};
}

// A tile of ROWS token rows by COLS columns (of which ncols hold data), fetched into
// registers and put into LDS later, so that the fetch runs behind other work.  Rows past
// `rows` and columns past `ncols` become zero and are not touched in memory.  WHOLE: ncols
// is a multiple of the vector, so a vector is there or not; those that are not are read at
// `base` (which must be readable) with no branch, and made zero when they are put: a select
// next to the read would wait for it there.
template <typename T, int ROWS, int COLS, int THREADS, bool WHOLE>
struct TileFetch {
    static constexpr int kPerRow = COLS / kVec<T>;
    static constexpr int kAll = ROWS * kPerRow, kCount = (kAll + THREADS - 1) / THREADS;
    u32x4 r[kCount];
    __device__ __forceinline__ static bool has(int k, int tid) { return kAll % THREADS == 0 || tid + k * THREADS < kAll; }
    __device__ __forceinline__ static int row_of(int k, int tid) { return (tid + k * THREADS) / kPerRow; }
    __device__ __forceinline__ static int col_of(int k, int tid) { return (tid + k * THREADS) % kPerRow * kVec<T>; }
    __device__ __forceinline__ void fetch(const T *__restrict__ base, int64_t stride, int rows, int ncols, int tid) {
#pragma unroll
        for (int k = 0; k < kCount; ++k) {
            const int row = row_of(k, tid), c = col_of(k, tid);
            const bool on = row < rows && has(k, tid);
            if constexpr (WHOLE) r[k] = *(const u32x4_a2 *)(base + (on && c < ncols ? row * stride + c : 0));
            else r[k] = load_vec<T>(base + (on ? row * stride + c : 0), on ? ncols - c : 0);
        }
    }
    // Vector k as it was fetched with these rows and ncols.
    __device__ __forceinline__ u32x4 get(int k, int rows, int ncols, int tid) const {
        if (!WHOLE) return r[k];
        return row_of(k, tid) < rows && col_of(k, tid) < ncols ? r[k] : u32x4{0, 0, 0, 0};
    }
    __device__ __forceinline__ void put(T *tile, int ld, int rows, int ncols, int tid) const {
#pragma unroll
        for (int k = 0; k < kCount; ++k)
            if (has(k, tid)) *(u32x4 *)(tile + row_of(k, tid) * ld + col_of(k, tid)) = get(k, rows, ncols, tid);
    }
};

}  // namespace seq
}  // namespace ddpm
