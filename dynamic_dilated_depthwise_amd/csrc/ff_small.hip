// ff_small.hip -- the backward through an activation or a gate of few channels (a feature map's pixels:
// up to 64 columns of x and 256 of z) in one pass over the rows:
//
//   z = x W^T + bias,  dz from z and grad,  grad_x = dz W,  grad_W += dz^T x,  grad_bias += sums of dz
//
// The weight stays in LDS, z and dz never leave the chip: a workgroup takes 64 rows at a time (float32:
// 32), makes their z (its waves 32 columns each), puts dz into LDS, and multiplies it by both; grad_W
// stays in registers until the workgroup's last rows and leaves as one row of float32 partials, which a
// second kernel adds up.  65536 rows of 64 to 2 128 take 36 us in bfloat16 and 52 in float32, 262144 rows 103
// and 169.  The bytes of 65536 rows alone are 6.5 us and 13.  What bounds it are vector instructions (47 % of the
// cycles of 262144 rows in bfloat16, 37 % in float32; the matrix units 23 % and 42 %), most of them the activation's
// slopes and the fragments' and rows' addresses, and eight waves a compute unit to hide the rest behind.
//
// Everything in LDS is bfloat16, of float32 three planes (see split_of), of bfloat16's dz two, each made once:
// split at every read the float32 kernel took 79 us for 65536 rows of 64 to 2 128, most of it vector
// instructions.  A sheet is ROWS rows of 128 bytes for each 64 columns, its 16-byte chunks placed by an exclusive
// or with bits of the row, such that fragments are read both along its rows and down its columns with few
// conflicts.
#include "ff_gemm.hpp"
#include "seq_launch.hpp"

namespace ddpm {
namespace ff {

namespace {

constexpr int kCols = kSmallCols, kWidth = kSmallWidth, kThreads = 512;
template <typename T> constexpr int kCopies = Elem<T>::is_bf16 ? 1 : kParts;  // planes of a sheet
template <typename T> constexpr int kTermsOfZ = Elem<T>::is_bf16 ? 2 : kParts;      // of dz's

// A lane's places in a sheet, made once a phase: those of its fragments differ by an exclusive or of a chunk's
// number with a constant below N and by constants that the instructions hold.
template <int N> struct Turned { int to[N]; };
// turn: uniform; by: bytes of a turn
template <int N> __device__ __forceinline__ Turned<N> turned(int sheet, int lane_at, int turn, int by) {
    Turned<N> r;
#pragma unroll
    for (int v = 0; v < N; ++v) r.to[v] = sheet + (lane_at ^ (turn ^ v) * by);
    return r;
}
// Row l16, column 8 g; a turn where 16 rows or 32 columns further.
__device__ __forceinline__ Turned<2> lanes_along(int sheet, int l16, int g, int turn) {
    return turned<2>(sheet, l16 * 128 + (((g ^ l16 ^ l16 / 8 * 2) & 7) << 4), turn, 64);
}
// Row 8 g + l16 / 4, column 4 (l16 % 4); a turn for 16 columns, two turns where four rows further.
__device__ __forceinline__ Turned<4> lanes_down(int sheet, int l16, int g, int turn) {
    return turned<4>(sheet, (8 * g + l16 / 4) * 128 + ((l16 % 4 / 2 ^ l16 / 4 ^ 2 * g) << 4) + l16 % 2 * 8, turn, 32);
}
// Row l16, column 4 g; a turn for 16 columns, two for 32 columns or 16 rows.
__device__ __forceinline__ Turned<4> lanes_put(int sheet, int l16, int g, int turn) {
    return turned<4>(sheet, l16 * 128 + (((g / 2 ^ l16 ^ l16 / 8 * 2) & 7) << 4) + g % 2 * 8, turn, 32);
}

template <typename T, int ROWS, int COLS, int PLANES = kCopies<T>>
struct Sheet {
    static constexpr int kPane = ROWS * 128, kPlane = COLS / 64 * kPane, kBytes = kPlane * PLANES;
    typedef std::conditional_t<PLANES == 1, bf16x8, Terms<PLANES>> Fragment;
    __device__ __forceinline__ static int bits(int row) { return (row ^ (row >> 3) << 1) & 7; }
    // Byte offset of column c of a row; eight neighbours stay together.
    __device__ __forceinline__ static int at(int row, int c) {
        return c / 64 * kPane + row * 128 + ((c % 64 / 8 ^ bits(row)) << 4) + c % 8 * 2;
    }
    // Four neighbours.
    __device__ __forceinline__ static void put4(char *to, f32x4 v) {
#pragma unroll
        for (int k = 0; k < PLANES; ++k) {
            u16x4 t;
#pragma unroll
            for (int e = 0; e < 4; ++e) t[e] = f32_to_bf16_bits(PLANES > 1 && k == 0 ? within_bf16(v[e]) : v[e]);
            *(u16x4 *)(to + k * kPlane) = t;
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] -= bf16_bits_to_f32(t[e]);
        }
    }
    // A 16-byte vector of T from column c.
    __device__ __forceinline__ static void put(char *p, int row, int c, const u32x4 &v) {
        if constexpr (Elem<T>::is_bf16) *(u32x4 *)(p + at(row, c)) = v;
        else put4(p + at(row, c), __builtin_bit_cast(f32x4, v));
    }
    // A fragment: index over the rows 16 t .., contraction over the columns 32 r ..; at: lanes_along of the sheet
    // (or of its rows from a t on, turned by t % 2, and then t counts from there).
    __device__ __forceinline__ static Fragment along(const char *lds, const Turned<2> &at, int t, int r) {
        const char *from = lds + at.to[(r ^ t) & 1] + t * 2048 + r / 2 * kPane;
        if constexpr (PLANES == 1) {
            return *(const bf16x8 *)from;
        } else {
            Fragment v;
#pragma unroll
            for (int k = 0; k < PLANES; ++k) v.part[k] = *(const bf16x8 *)(from + k * kPlane);
            return v;
        }
    }
    // Index over the columns 16 t .., contraction over the rows 32 r ..; at: lanes_down of the sheet (or of
    // its columns from a t on, turned by t % 4).
    __device__ __forceinline__ static Fragment down(const char *lds, const Turned<4> &at, int t, int r) {
        typedef __attribute__((address_space(3))) s16x4 *lds_ptr;
        const char *first = lds + at.to[t] + r * 4096, *second = lds + at.to[t ^ 2] + 512 + r * 4096;
        bf16x8 v[PLANES];
#pragma unroll
        for (int k = 0; k < PLANES; ++k) {
            const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(first + k * kPlane));
            const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(second + k * kPlane));
            u16x8 u;
#pragma unroll
            for (int e = 0; e < 4; ++e) { u[e] = (uint16_t)a[e]; u[4 + e] = (uint16_t)b[e]; }
            v[k] = __builtin_bit_cast(bf16x8, u);
        }
        if constexpr (PLANES == 1) return v[0];
        else if constexpr (PLANES == 2) return Fragment{{v[0], v[1]}};
        else return Fragment{{v[0], v[1], v[2]}};
    }
};

template <typename T> struct Small {
    static constexpr int kRows = small_rows(Elem<T>::is_bf16), kXs = Elem<T>::is_bf16 ? 2 : 1;  // x: being read, being put
    typedef Sheet<T, kWidth, kCols> W;
    typedef Sheet<T, kRows, kCols> X;
    typedef Sheet<T, kRows, kWidth, kTermsOfZ<T>> Z;
    static constexpr int kLds = W::kBytes + kXs * X::kBytes + Z::kBytes;
    static constexpr int kPer = kVec<T>, kXChunks = kRows * kCols / kPer / kThreads, kWChunks = kWidth * kCols / kPer / kThreads;
    static constexpr int kM = kRows / 16, kOwn = 4 * kM / 8;  // sixteens of rows; of a wave's in grad_x
};
static_assert(Small<float>::kLds <= 160 * 1024, "one compute unit's LDS");
static_assert(Small<bf16_t>::kLds <= 160 * 1024, "one compute unit's LDS");

// Row of W that is row n of its sheet: gated, 16 of the gate's, the same 16 of the other half, and so on.
template <bool GATED>
__device__ __forceinline__ int column_of(int n) { return GATED ? (n >> 5 << 4) + (n & 15) : n; }

template <typename T, bool GATED>
__global__ __launch_bounds__(kThreads, 2) void small_backward_kernel(const SmallBackward a) {
    typedef Small<T> S;
    extern __shared__ __attribute__((aligned(16))) char lds[];
    constexpr int w = 0, x = S::W::kBytes, dz = x + S::kXs * S::X::kBytes;  // where in LDS
    const int tid = threadIdx.x, wave = wave_of(tid), lane = tid % kWave, l16 = lane % 16, g = lane / 16;
    const int C = a.C, N = a.N;
    constexpr int kRows = S::kRows, kM = S::kM, kOwn = S::kOwn;
    const int64_t tiles = (a.rows + kRows - 1) / kRows;

    // chunk i of the thread: (row, column) of a sheet
    const auto row_of = [&](int i) { return (i * kThreads + tid) / (kCols / S::kPer); };
    const auto col_of = [&](int i) { return (i * kThreads + tid) % (kCols / S::kPer) * S::kPer; };
#pragma unroll
    for (int i = 0; i < S::kWChunks; ++i) {
        const int n = row_of(i), c = col_of(i), f = column_of<GATED>(n);
        const int64_t from = f + (GATED && n & 16 ? N : 0);
        const bool on = f < N && c < C;
        S::W::put(lds + w, n, c, load_vec<T>((const T *)a.weight + (on ? from * a.weight_ld + c : 0), on ? C - c : 0));
    }
    u32x4 xn[S::kXChunks];
    const auto fetch = [&](int64_t tile) {
#pragma unroll
        for (int i = 0; i < S::kXChunks; ++i) {
            const int c = col_of(i);
            const int64_t m = tile * kRows + row_of(i);
            const bool on = m < a.rows && c < C;
            xn[i] = load_vec<T>((const T *)a.x + (on ? m * a.x_ld + c : 0), on ? C - c : 0);
        }
    };
    const auto put = [&](char *to) {
#pragma unroll
        for (int i = 0; i < S::kXChunks; ++i) S::X::put(to, row_of(i), col_of(i), xn[i]);
    };
    f32x4 gw[4][2], sum[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        sum[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) gw[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    fetch(blockIdx.x);
    put(lds + x);
    int now = 0;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x, now ^= S::kXs - 1) {
        __syncthreads();  // x is there, and dz is read
        const int xt = x + now * S::X::kBytes;
        const int64_t m0 = tile * kRows;
        const int left = (int)(a.rows - m0 < kRows ? a.rows - m0 : kRows);
        if (tile + gridDim.x < tiles) fetch(tile + gridDim.x);
        const auto grad_of = [&](int m, int f_, int n) {
            f32x4 gr = {0.f, 0.f, 0.f, 0.f};
            const T *grad = (const T *)a.grad + (n > 0 ? (m0 + m) * a.grad_ld + f_ : 0);
            if (n >= 4) {
                gr = load_four<T>(grad);
            } else {
#pragma unroll
                for (int e = 0; e < 3; ++e)
                    if (e < n) gr[e] = Elem<T>::to_f32(grad[e]);
            }
            return gr;
        };
        // Before z is made in float32 (262144 rows of 64 to 2 128: 202 us, so 184); bfloat16 gains nothing (103 us,
        // so 104; of 64 to 256 145 and 154).
        constexpr bool kAhead = !Elem<T>::is_bf16;
        f32x4 ahead[2][kAhead ? kM : 1];
        if constexpr (kAhead) {
#pragma unroll
            for (int h = 0; h < (GATED ? 1 : 2); ++h)
#pragma unroll
                for (int j = 0; j < kM; ++j) {
                    const int m = 16 * j + l16, at = column_of<GATED>(32 * wave + 16 * h) + 4 * g;
                    ahead[h][j] = grad_of(m, at, m < left ? N - at : 0);
                }
        }
        // z: 32 columns of the wave's by 64 rows
        f32x4 z[2][kM];
        const Turned<2> at_x = lanes_along(xt, l16, g, 0), at_w = lanes_along(w + wave * 4096, l16, g, 0);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < kM; ++j) z[h][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int r = 0; r < kCols / 32; ++r) {
            Operand<T> q[kM];
#pragma unroll
            for (int j = 0; j < kM; ++j) q[j] = S::X::along(lds, at_x, j, r);
#pragma unroll
            for (int h = 0; h < 2; ++h) multiply<kM>(z[h], S::W::along(lds, at_w, h, r), q);
        }
        // dz, in bfloat16 as two terms (one would make the gradients' error 1.4 times that of their own rounding).
        // The wave's two sixteens of z's columns, in the sheet's order, are a gate's
        // and its other half's, or neighbours; a lane has four of each.
        const Turned<4> at_put = lanes_put(dz + wave / 2 * S::Z::kPane, l16, g, wave % 2 * 2);
        int f[2];
        f32x4 bias[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            f[h] = column_of<GATED>(32 * wave + 16 * h) + 4 * g;
            bias[h] = load4(a.bias + (f[h] < N ? (GATED && h ? N : 0) + f[h] : 0), f[h] < N ? N - f[h] : 0);
        }
#pragma unroll
        for (int j = 0; j < kM; ++j) {
            const int m = 16 * j + l16;
            f32x4 d[2];
#pragma unroll
            for (int h = 0; h < (GATED ? 1 : 2); ++h) {
                const int n = m < left ? N - f[h] : 0;
                const f32x4 gr = kAhead ? ahead[h][kAhead ? j : 0] : grad_of(m, f[h], n);
                float v[4], s[4], t[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) t[e] = z[h][j][e] + bias[h][e];
                slopes(t, v, s, a.act);
#pragma unroll
                for (int e = 0; e < 4; ++e) {  // nothing of columns and rows that are not there, whatever their z
                    const float other = GATED ? z[1][j][e] + bias[1][e] : 1.f;
                    d[h][e] = e < n ? gr[e] * other * s[e] : 0.f;
                    if constexpr (GATED) d[1][e] = e < n ? gr[e] * v[e] : 0.f;
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) S::Z::put4(lds + at_put.to[h ^ j % 2 * 2] + j * 2048, d[h]);
        }
        __syncthreads();
        // grad_x: 16 columns of C by 32 rows a wave (float32: 16)
        if (a.grad_x != nullptr) {
            f32x4 gx[kOwn];
            const int t = wave % 4, j0 = wave / 4 * kOwn;
            const Turned<2> at_z = lanes_along(dz + j0 * 2048, l16, g, j0 % 2);
            const Turned<4> at_wd = lanes_down(w, l16, g, t);
#pragma unroll
            for (int j = 0; j < kOwn; ++j) gx[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int r = 0; r < kWidth / 32; ++r) {
                typename S::Z::Fragment q[kOwn];
#pragma unroll
                for (int j = 0; j < kOwn; ++j) q[j] = S::Z::along(lds, at_z, j, r);
                multiply<kOwn>(gx, S::W::down(lds, at_wd, 0, r), q);
            }
            const int c = 16 * t + 4 * g;
#pragma unroll
            for (int j = 0; j < kOwn; ++j) {
                const int m = 16 * (j0 + j) + l16;
                if (m < left && c < C) store4<T>((T *)a.grad_x + (m0 + m) * C + c, gx[j], C - c);
            }
        }
        // grad_W: all columns of C by the wave's 32 of z
        if (a.part != nullptr) {
            const Turned<4> at_z = lanes_down(dz + wave / 2 * S::Z::kPane, l16, g, wave % 2 * 2), at_xd = lanes_down(xt, l16, g, 0);
#pragma unroll
            for (int r = 0; r < kRows / 32; ++r) {
                const typename S::Z::Fragment q[2] = {S::Z::down(lds, at_z, 0, r), S::Z::down(lds, at_z, 1, r)};
                add_up<2>(sum, q);
#pragma unroll
                for (int i = 0; i < 4; ++i) multiply<2>(gw[i], S::X::down(lds, at_xd, i, r), q);
            }
        }
        if (tile + gridDim.x < tiles) {
            if constexpr (S::kXs == 1) __syncthreads();  // x is read
            put(lds + x + (now ^ (S::kXs - 1)) * S::X::kBytes);
        }
    }
    if (a.part != nullptr) {
        const int64_t width = GATED ? 2 * N : N;
        float *part = a.part + blockIdx.x * (width * C + width);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int n = column_of<GATED>(32 * wave + 16 * j) + l16;
            const int64_t row = n + (GATED && j ? N : 0);
            if (n >= N) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (16 * i + 4 * g < C) store4<float>(part + row * C + 16 * i + 4 * g, gw[i][j], C - 16 * i - 4 * g);
            if (g == 0) part[width * C + row] = sum[j][0];
        }
    }
}

template <typename T, bool GATED>
hipError_t run(SmallBackward a, hipStream_t stream) {
    const auto kernel = small_backward_kernel<T, GATED>;
    const hipError_t e = hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, Small<T>::kLds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3(small_groups(a.rows, Elem<T>::is_bf16)), dim3(kThreads), Small<T>::kLds, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_small_backward(bool gated, SmallBackward a, void *grad_weight, void *grad_bias, bool bf16, hipStream_t stream) {
    const hipError_t e = bf16 ? gated ? run<bf16_t, true>(a, stream) : run<bf16_t, false>(a, stream)
                              : gated ? run<float, true>(a, stream) : run<float, false>(a, stream);
    if (e != hipSuccess || a.part == nullptr) return e;
    const int64_t width = gated ? 2 * a.N : a.N;
    return seq::launch_sum_rows(a.part, small_groups(a.rows, bf16), width * a.C, width, grad_weight, grad_bias, bf16, stream);
}

}  // namespace ff
}  // namespace ddpm
