// linattn_walk.hip -- linear attention with a decay for each head, over whole sequences.
//
// For a value head with decay a, S_t = a S_{t-1} + k_t^T v_t and o_t = q_t S_t. Over a chunk of
// 64 rows entered with the state S (row r of the chunk, n rows):
//     o_r = sum_{j <= r} a^(r-j) (q_r . k_j) v_j + a^(r+1) q_r S
//     S  <- a^n S + sum_j a^(n-1-j) k_j^T v_j
// so a chunk is four small matrix products, and the state passes from chunk to chunk in
// registers. The gradients are the same walk with other operands (dq: the rows do, v, k; and
// backwards in time dk: v, do, q; dv: k, q, do).
//
// A workgroup of four waves walks one segment of a sequence for one value head and one block of
// value channels; a wave owns NV of them, with all DK key channels of their state. Every product
// is laid out so that what one leaves in registers is what the next takes:
//   * the state as S[m = key][n = value channel] (a lane holds one value channel, four
//     consecutive keys a tile) is the left operand of o^T = S^T q^T, and
//   * v read from LDS by the transposing loads (a lane holds one value channel, eight
//     consecutive rows) serves o^T = v^T p^T from the left and S = k^T v from the right.
// Only p = (q k^T with its decays) goes through LDS, wave w computing rows 16w .. 16w + 15.
#include "../../include/cconv.h"
#include "cconv_device.hpp"
#include "linattn_internal.hpp"

namespace cconv {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Four rows by sixteen columns of LDS, transposed: within each group of 16 lanes, lane i points
// at row i/4, columns 4*(i%4) ..; it receives column i of the four rows.
__device__ __forceinline__ u32x2 load_tr(const uint16_t* p) {
    using L = __attribute__((address_space(3))) s16x4;
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((L*)(p)));
}

// a^n for the decay's base-2 logarithm; a^0 = 1 also where a = 0.
__device__ __forceinline__ float power(float g2, int n) { return n == 0 ? 1.0f : __builtin_amdgcn_exp2f(g2 * static_cast<float>(n)); }

// The same for a span of rows that may be long: the exponent's product in 64 bits.
__device__ __forceinline__ float power_long(float g, int64_t n) {
    return n == 0 ? 1.0f
                  : __builtin_amdgcn_exp2f(static_cast<float>(static_cast<double>(g) * static_cast<double>(n) * 1.4426950408889634));
}

// Byte offset that lies outside every buffer range below: a load from it gives zeros, a store to it
// is dropped.
constexpr uint32_t kNowhere = 0x80000000u;
constexpr int kRange = 0x7fffffff;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t chunk_rsrc(const void* p) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, kRange, 0x00020000);
}

// Eight channels of a row, of which the first `have` exist (VEC = 8: all or, at kNowhere, none). No
// branches, so a chunk's loads are issued back to back and stay in flight.
template <int VEC>
__device__ __forceinline__ u32x4 load8(__amdgpu_buffer_rsrc_t r, uint32_t off, int soff, int have) {
    if constexpr (VEC == 8) {
        return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, soff, 0));
    } else if constexpr (VEC == 4) {
        const u32x2 x = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, off, soff, 0));
        const u32x2 y = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, have > 4 ? off + 8 : kNowhere, soff, 0));
        return u32x4{x.x, x.y, y.x, y.y};
    } else {
        uint32_t e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            e[i] = static_cast<uint16_t>(__builtin_amdgcn_raw_buffer_load_b16(r, i < have ? off + 2 * i : kNowhere, soff, 0));
        return u32x4{e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16};
    }
}

// One operand's part in the staging of a chunk: 256 threads, eight channels each, COLS (padded)
// channels a row. The chunk is addressed from its lowest row in memory: its first row, or, walked
// backwards, its 64th (which may lie before the sequence: rows past the end are never read).
template <int COLS, int VEC>
struct Stage {
    static constexpr int kPerRow = COLS / 8, kRows = 256 / kPerRow, kPasses = kChunk / kRows, kPitch = COLS + 8;
    u32x4 r[kPasses];
    const uint16_t* p;  // lowest row of the next chunk
    int64_t step;       // elements from a chunk to the next
    int pass;           // bytes between a thread's rows of two passes (first row to last of the chunk, upwards)
    int row, have;      // the thread's row in pass 0 and its channels
    uint32_t off;
    bool up;

    __device__ __forceinline__ void open(const uint16_t* first_row, const Rows& x, bool reverse, int col0) {
        row = threadIdx.x / kPerRow;
        const int col = col0 + (threadIdx.x % kPerRow) * 8;
        have = x.dim - col;
        up = !reverse;
        p = reverse ? first_row - (kChunk - 1) * x.st : first_row;
        step = reverse ? -kChunk * x.st : kChunk * x.st;
        const int st = static_cast<int>(x.st);
        pass = kRows * st * 2;
        off = have <= 0 ? kNowhere : static_cast<uint32_t>(((reverse ? kRows - 1 - row : row) * st + col) * 2);
    }
    __device__ __forceinline__ void load(int n) {
        const __amdgpu_buffer_rsrc_t b = chunk_rsrc(p);
#pragma unroll
        for (int i = 0; i < kPasses; ++i)
            r[i] = load8<VEC>(b, row + i * kRows < n ? off : kNowhere, (up ? i : kPasses - 1 - i) * pass, have);
        p += step;
    }
    __device__ __forceinline__ void store(uint16_t* lds) {
        uint16_t* d = lds + row * kPitch + (threadIdx.x % kPerRow) * 8;
#pragma unroll
        for (int i = 0; i < kPasses; ++i) *reinterpret_cast<u32x4*>(d + i * kRows * kPitch) = r[i];
    }
};

__device__ __forceinline__ bool finite(float x) { return __builtin_fabsf(x) <= 3.402823466e38f; }

}  // namespace

template <int DK, int NV, int VEC, bool STATES>
__global__ __launch_bounds__(256, 2) void cconv_linattn_walk_kernel(WalkArgs a) {
    constexpr int DVB = 4 * NV, NM = NV / 16, NT = DK / 16, NK = DK / 32;
    constexpr int PK = DK + 8, PV = DVB + 8, PP = kChunk + 8;
    __shared__ __align__(16) uint16_t lk[kChunk * PK];
    __shared__ __align__(16) uint16_t lv[kChunk * PV];
    __shared__ __align__(16) uint16_t lq[STATES ? 8 : kChunk * PK];
    __shared__ __align__(16) uint16_t lp[STATES ? 8 : kChunk * PP];

    if (a.status && *a.status != CCONV_OK) return;
    const uint32_t tile = static_cast<uint32_t>(xcd_tile(blockIdx.x, gridDim.x)), per_seg = static_cast<uint32_t>(a.vblocks * a.HV);
    const uint32_t hvb = tile % per_seg;
    const int vb = static_cast<int>(hvb % a.vblocks), hv = static_cast<int>(hvb / a.vblocks);
    const int64_t seg = tile / per_seg;
    int64_t seq, start, len, first;  // the segment's sequence, its rows, and the segment's first row in it
    if (a.cu) {
        seq = a.seg_of[2 * seg];
        if (seq < 0) return;
        first = static_cast<int64_t>(a.seg_of[2 * seg + 1]) * a.seg_rows;
        start = a.cu[seq];
        len = a.cu[seq + 1] - start;
    } else {
        seq = static_cast<uint32_t>(seg) / static_cast<uint32_t>(a.segs);
        first = (seg - seq * a.segs) * a.seg_rows;
        start = 0;
        len = a.T;
    }
    const bool last = first + a.seg_rows >= len;
    if (STATES && last) return;
    const int64_t rows = last ? len - first : a.seg_rows;
    const int64_t batch = a.cu ? 0 : seq;

    const int wave = wave_id(), lane = threadIdx.x % kWave, i16 = lane % 16, g = lane / 16;
    const float g2 = a.log_decay[hv] * 1.4426950408889634f;
    const float aC = power(g2, kChunk);

    // rows are taken in the walk's order: backwards from the last row when reversed
    const int64_t row0 = start + (a.reverse ? len - 1 - first : first);
    auto base = [&](const Rows& x) { return x.p + batch * x.sb + row0 * x.st + (hv / x.hdiv) * x.sh; };
    Stage<DK, VEC> sk;
    Stage<DVB, VEC> sv;
    Stage<STATES ? 64 : DK, VEC> sq;
    sk.open(base(a.k), a.k, a.reverse, 0);
    sv.open(base(a.v), a.v, a.reverse, vb * DVB);
    if constexpr (!STATES) sq.open(base(a.q), a.q, a.reverse, 0);

    int n = static_cast<int>(rows < kChunk ? rows : kChunk);
    sk.load(n);
    sv.load(n);
    if constexpr (!STATES) sq.load(n);

    // the state: S[t][m] holds keys 16t + 4g + 0..3 of value channel dv0 + 16m + i16
    const int dv0 = vb * DVB + wave * NV;
    f32x4 S[NT][NM];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int m = 0; m < NM; ++m) S[t][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int64_t frag = (static_cast<int64_t>(hv) * a.vblocks + vb) * DK * DVB + (wave * 64 + lane) * 4;
    const int64_t seg_floats = static_cast<int64_t>(a.HV) * a.vblocks * DK * DVB;
    const int64_t matrix = (seq * a.HV + hv) * static_cast<int64_t>(a.k.dim) * a.v.dim;
    if constexpr (!STATES) {
        if (first > 0) {
            const float* c = a.states + (seg - 1) * seg_floats + frag;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int m = 0; m < NM; ++m) S[t][m] = *reinterpret_cast<const f32x4*>(c + (t * NM + m) * 1024);
        }
        if (a.init) {
            const float w = power_long(a.log_decay[hv], first);
            const __amdgpu_buffer_rsrc_t ib = chunk_rsrc(a.init + matrix);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int m = 0; m < NM; ++m)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int dk = 16 * t + 4 * g + r, dv = dv0 + 16 * m + i16;
                        const uint32_t at = dk < a.k.dim && dv < a.v.dim ? 4 * (dk * a.sk + dv * a.sv) : kNowhere;
                        S[t][m][r] = __builtin_fmaf(w, __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(ib, at, 0, 0)), S[t][m][r]);
                    }
        }
    }

    // decays that stay the same from chunk to chunk
    float near[4], far[4], carry[4];  // p's diagonal tile; p's tiles below, less 16 rows a tile; rows 16b + i16
    if constexpr (!STATES) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int d = i16 - 4 * g - r;
            near[r] = a.alpha * power(g2, d < 0 ? 0 : d);
            far[r] = a.alpha * power(g2, 16 + d);
            carry[r] = a.beta * power(g2, 16 * r + i16 + a.shift);
        }
        // p's tiles above the diagonal are read by the 32-row products and stay zero
        for (int i = threadIdx.x; i < kChunk * PP / 2; i += 256) reinterpret_cast<uint32_t*>(lp)[i] = 0u;
    }
    float late[8];  // row 8g + e of a full chunk's second half
#pragma unroll
    for (int e = 0; e < 8; ++e) late[e] = a.gamma * power(g2, 32 - a.shift - 8 * g - e);
    const float early = power(g2, 32);

    for (int64_t c0 = 0; c0 < rows; c0 += kChunk) {
        lds_barrier();  // the chunk before has been read
        sk.store(lk);
        sv.store(lv);
        if constexpr (!STATES) sq.store(lq);
        lds_barrier();
        const int left = static_cast<int>(rows - c0 < 2 * kChunk ? rows - c0 : 2 * kChunk);
        n = left < kChunk ? left : kChunk;
        if (left > kChunk) {
            sk.load(left - kChunk);
            sv.load(left - kChunk);
            if constexpr (!STATES) sq.load(left - kChunk);
        }
        u32x4 vf[2][NM];  // value channel dv0 + 16m + i16, rows 32h + 8g + 0..7
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int m = 0; m < NM; ++m) {
                const uint16_t* p = lv + (32 * h + 8 * g + i16 / 4) * PV + wave * NV + 16 * m + 4 * (i16 % 4);
                const u32x2 lo = load_tr(p), hi = load_tr(p + 4 * PV);
                vf[h][m] = u32x4{lo.x, lo.y, hi.x, hi.y};
            }

        if constexpr (!STATES) {
            // p^T = k q^T, rows 16*wave + i16 of q
            u32x4 qf[NK];
#pragma unroll
            for (int kk = 0; kk < NK; ++kk)
                qf[kk] = *reinterpret_cast<const u32x4*>(lq + (16 * wave + i16) * PK + 32 * kk + 8 * g);
            float down = 1.0f;  // a^(16 * (tiles between))
            const float a16 = power(g2, 16);
#pragma unroll
            for (int back = 0; back < 4; ++back) {
                const int jb = wave - back;
                if (jb >= 0) {
                    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int kk = 0; kk < NK; ++kk)
                        acc = mfma(*reinterpret_cast<const u32x4*>(lk + (16 * jb + i16) * PK + 32 * kk + 8 * g), qf[kk], acc);
                    float p[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        if (back == 0)  // a later row's product is dropped, whatever it holds
                            p[r] = i16 >= 4 * g + r ? acc[r] * near[r] : 0.0f;
                        else
                            p[r] = acc[r] * (far[r] * down);
                    }
                    if (back > 0) down *= a16;
                    *reinterpret_cast<u32x2*>(lp + (16 * wave + i16) * PP + 16 * jb + 4 * g) =
                        u32x2{pack_bf16x2(p[0], p[1]), pack_bf16x2(p[2], p[3])};
                }
            }
            // o^T = S^T q^T: the state rounded to bf16 as a matrix operand (a relative 2^-9 of each
            // entry, as the products' other operand has; the state itself stays in 32 bits)
            f32x4 O[4][NM];
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
                for (int m = 0; m < NM; ++m) O[b][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int kk = 0; kk < NK; ++kk) {
                u32x4 sf[NM];
#pragma unroll
                for (int m = 0; m < NM; ++m) {
                    const f32x4 x = S[2 * kk][m], y = S[2 * kk + 1][m];
                    sf[m] = u32x4{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(y[0], y[1]),
                                  pack_bf16x2(y[2], y[3])};
                }
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const uint16_t* p = lq + (16 * b + i16) * PK + 32 * kk + 4 * g;
                    const u32x2 lo = *reinterpret_cast<const u32x2*>(p), hi = *reinterpret_cast<const u32x2*>(p + 16);
                    const u32x4 qt = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
                    for (int m = 0; m < NM; ++m) O[b][m] = mfma(sf[m], qt, O[b][m]);
                }
            }
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
                for (int m = 0; m < NM; ++m)
#pragma unroll
                    for (int r = 0; r < 4; ++r) O[b][m][r] *= carry[b];
            lds_barrier();  // p is whole
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                f32x4 enter[NM];
                float sum = 0.0f;
#pragma unroll
                for (int m = 0; m < NM; ++m) enter[m] = O[b][m];
#pragma unroll
                for (int h = 0; h <= b / 2; ++h) {
                    const u32x4 pf = *reinterpret_cast<const u32x4*>(lp + (16 * b + i16) * PP + 32 * h + 8 * g);
#pragma unroll
                    for (int m = 0; m < NM; ++m) O[b][m] = mfma(vf[h][m], pf, O[b][m]);
                }
#pragma unroll
                for (int m = 0; m < NM; ++m)
#pragma unroll
                    for (int r = 0; r < 4; ++r) sum = __builtin_fmaf(O[b][m][r], 0.0f, sum);
                // An infinity or NaN in a later row of v meets p's zeros above the diagonal and would make
                // NaN of rows that do not depend on it: such rows are summed again without them.
                if (__builtin_expect(__builtin_amdgcn_ballot_w64(sum != 0.0f) != 0, 0)) {
#pragma unroll
                    for (int m = 0; m < NM; ++m) O[b][m] = enter[m];
#pragma clang loop unroll(disable)
                    for (int j = 0; j <= 16 * b + i16; ++j) {
                        const float pj = bf16_lo(lp[(16 * b + i16) * PP + j]);
#pragma unroll
                        for (int m = 0; m < NM; ++m)
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                O[b][m][r] = __builtin_fmaf(pj, bf16_lo(lv[j * PV + wave * NV + 16 * m + 4 * g + r]), O[b][m][r]);
                    }
                }
            }
            // rows of o, addressed like the operands' from the chunk's lowest row
            const int es = a.o_f32 ? 4 : 2, ost = static_cast<int>(a.o_st) * es;
            const int64_t low = row0 + (a.reverse ? -(c0 + kChunk - 1) : c0);
            const __amdgpu_buffer_rsrc_t ob =
                chunk_rsrc(static_cast<char*>(a.o) + (batch * a.o_sb + low * a.o_st + hv * a.o_sh) * es);
            const uint32_t o0 = static_cast<uint32_t>((a.reverse ? 15 - i16 : i16) * ost + (dv0 + 4 * g) * es);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int sb = (a.reverse ? 3 - b : b) * 16 * ost;
                const bool in = 16 * b + i16 < n;
#pragma unroll
                for (int m = 0; m < NM; ++m) {
                    const int dv = dv0 + 16 * m + 4 * g;
                    const uint32_t at = in && dv < a.v.dim ? o0 + 16 * m * es : kNowhere;
                    const u32x2 w = {pack_bf16x2(O[b][m][0], O[b][m][1]), pack_bf16x2(O[b][m][2], O[b][m][3])};
                    if (a.o_vec == 4) {
                        if (a.o_f32)
                            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, O[b][m]), ob, at, sb, 0);
                        else
                            __builtin_amdgcn_raw_buffer_store_b64(w, ob, at, sb, 0);
                    } else {
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const uint32_t e = dv + r < a.v.dim ? at + r * es : kNowhere;
                            if (a.o_f32)
                                __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(O[b][m][r]), ob, e, sb, 0);
                            else
                                __builtin_amdgcn_raw_buffer_store_b16(static_cast<uint16_t>(w[r / 2] >> (16 * (r % 2))), ob, e, sb, 0);
                        }
                    }
                }
            }
        }

        // S = a^n S + k^T (a^(n-shift-j) v): the weighted v as a sum of two bf16 values (the second
        // holds what the first rounds off), so the state keeps about 17 bits of every term
        const float an = n == kChunk ? aC : power(g2, n);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int m = 0; m < NM; ++m)
#pragma unroll
                for (int r = 0; r < 4; ++r) S[t][m][r] *= an;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = h == 0 ? late[e] * early : late[e];
            if (n < kChunk) {  // rows past the end hold zeros; their weight only has to be finite
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int left_rows = n - a.shift - 32 * h - 8 * g - e;
                    w[e] = a.gamma * power(g2, left_rows < 0 ? 0 : left_rows);
                }
            }
            u32x4 hi[NM], lo[NM];
#pragma unroll
            for (int m = 0; m < NM; ++m) {
                uint32_t x[4], y[4];
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    const float u0 = bf16_lo(vf[h][m][d]) * w[2 * d], u1 = bf16_hi(vf[h][m][d]) * w[2 * d + 1];
                    x[d] = pack_bf16x2(u0, u1);
                    const float l0 = u0 - bf16_lo(x[d]), l1 = u1 - bf16_hi(x[d]);
                    y[d] = pack_bf16x2(finite(l0) ? l0 : 0.0f, finite(l1) ? l1 : 0.0f);
                }
                hi[m] = u32x4{x[0], x[1], x[2], x[3]};
                lo[m] = u32x4{y[0], y[1], y[2], y[3]};
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const uint16_t* p = lk + (32 * h + 8 * g + i16 / 4) * PK + 16 * t + 4 * (i16 % 4);
                const u32x2 k0 = load_tr(p), k1 = load_tr(p + 4 * PK);
                const u32x4 kf = {k0.x, k0.y, k1.x, k1.y};
#pragma unroll
                for (int m = 0; m < NM; ++m) {
                    S[t][m] = mfma(kf, lo[m], S[t][m]);
                    S[t][m] = mfma(kf, hi[m], S[t][m]);
                }
            }
        }
    }

    if constexpr (STATES) {
        float* c = a.states + seg * seg_floats + frag;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int m = 0; m < NM; ++m) *reinterpret_cast<f32x4*>(c + (t * NM + m) * 1024) = S[t][m];
    } else if (last && a.fin) {
        const __amdgpu_buffer_rsrc_t fb = chunk_rsrc(a.fin + matrix);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int m = 0; m < NM; ++m)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int dk = 16 * t + 4 * g + r, dv = dv0 + 16 * m + i16;
                    const uint32_t at = dk < a.k.dim && dv < a.v.dim ? 4 * (dk * a.sk + dv * a.sv) : kNowhere;
                    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[t][m][r]), fb, at, 0, 0);
                }
    }
}

// One workgroup per (sequence, head, 1024 floats): the running sum over the sequence's segments.
__global__ __launch_bounds__(256) void cconv_linattn_scan_kernel(ScanArgs a) {
    if (a.status && *a.status != CCONV_OK) return;
    const int64_t parts = a.floats / 1024;
    const int64_t part = blockIdx.x % parts, hv = blockIdx.x / parts % a.HV, seq = blockIdx.x / (parts * a.HV);
    int64_t s0, s1;
    if (a.seq_seg) {
        s0 = a.seq_seg[seq], s1 = a.seq_seg[seq + 1];
    } else {
        s0 = seq * a.segs, s1 = s0 + a.segs;
    }
    const float w = power_long(a.log_decay[hv], a.seg_rows);
    f32x4* p = reinterpret_cast<f32x4*>(a.states + (s0 * a.HV + hv) * a.floats + part * 1024) + threadIdx.x;
    const int64_t step = a.HV * a.floats / 4;
    f32x4 c = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t s = s0; s + 1 < s1; ++s, p += step) {
        const f32x4 x = *p;
#pragma unroll
        for (int r = 0; r < 4; ++r) c[r] = __builtin_fmaf(w, c[r], x[r]);
        *p = c;
    }
}

// One block: the offsets' verdict, then a running sum of the sequences' segment counts, then
// (a wave per sequence) each segment's sequence and place in it. Entries past the last segment
// get sequence -1.
__global__ __launch_bounds__(1024) void cconv_linattn_plan_kernel(const int32_t* cu, int64_t nseq, int64_t total,
                                                                  int64_t seg_rows, int32_t* status, int32_t* seq_seg,
                                                                  int32_t* seg_of, int64_t segments) {
    __shared__ int32_t sum[16];
    __shared__ int32_t carry;
    bool bad = false;
    for (int64_t i = threadIdx.x; i < nseq; i += blockDim.x)
        if (cu[i] > cu[i + 1]) bad = true;
    if (threadIdx.x == 0 && (cu[0] != 0 || static_cast<int64_t>(cu[nseq]) != total)) bad = true;
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) {
        status[0] = bad ? CCONV_ERR_INDEX : CCONV_OK;
        carry = 0;
    }
    if (bad) return;
    __syncthreads();
    const int lane = threadIdx.x % kWave, wave = wave_id();
    for (int64_t base = 0; base < nseq; base += blockDim.x) {
        const int64_t i = base + threadIdx.x;
        int32_t c = 0;
        if (i < nseq) {
            const int64_t len = static_cast<int64_t>(cu[i + 1]) - cu[i];
            c = static_cast<int32_t>(len == 0 ? 1 : (len + seg_rows - 1) / seg_rows);
        }
        int32_t x = c;  // running sum over the wave
        for (int d = 1; d < kWave; d *= 2) {
            const int32_t y = __shfl_up(x, d);
            if (lane >= d) x += y;
        }
        if (lane == kWave - 1) sum[wave] = x;
        __syncthreads();
        int32_t before = carry;
        for (int w = 0; w < wave; ++w) before += sum[w];
        if (i < nseq) seq_seg[i] = before + x - c;
        __syncthreads();
        if (threadIdx.x == blockDim.x - 1) carry = before + x;
        __syncthreads();
    }
    const int32_t used = carry;
    if (threadIdx.x == 0) seq_seg[nseq] = used;
    __threadfence_block();
    __syncthreads();
    for (int64_t i = wave; i < nseq; i += blockDim.x / kWave) {
        const int32_t s0 = seq_seg[i], s1 = seq_seg[i + 1];
        for (int32_t s = s0 + lane; s < s1; s += kWave) {
            seg_of[2 * static_cast<int64_t>(s)] = static_cast<int32_t>(i);
            seg_of[2 * static_cast<int64_t>(s) + 1] = s - s0;
        }
    }
    for (int64_t s = used + threadIdx.x; s < segments; s += blockDim.x) seg_of[2 * s] = -1;
}

__global__ __launch_bounds__(256) void cconv_linattn_group_sum_kernel(GroupSumArgs a) {
    if (a.status && *a.status != CCONV_OK) return;
    const int64_t total = a.B * a.T * a.H * a.dim;
    for (int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; e < total; e += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t c = e % a.dim, h = e / a.dim % a.H, row = e / (static_cast<int64_t>(a.dim) * a.H);
        const float* p = a.part + (row * a.H + h) * a.grp * a.dim + c;
        float s = p[0];
        for (int g = 1; g < a.grp; ++g) s += p[static_cast<int64_t>(g) * a.dim];
        a.out[row / a.T * a.o_sb + row % a.T * a.o_st + h * a.o_sh + c] = static_cast<uint16_t>(pack_bf16x2(s, 0.0f) & 0xffffu);
    }
}

WalkShape walk_shape(int64_t Dk, int64_t Dv) {
    WalkShape w;
    w.DK = Dk <= 64 ? 64 : Dk <= 128 ? 128 : 256;
    // 256 keys: 16 value channels a wave keep the state at 64 registers
    w.NV = (w.DK <= 128 && Dv > 64) ? 32 : 16;
    return w;
}

template <int DK, int NV, int VEC>
static hipError_t walk_go(bool states, const WalkArgs& a, hipStream_t s) {
    const dim3 grid(static_cast<uint32_t>(a.segments * a.HV * a.vblocks)), block(256);
    if (states)
        hipLaunchKernelGGL((cconv_linattn_walk_kernel<DK, NV, VEC, true>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((cconv_linattn_walk_kernel<DK, NV, VEC, false>), grid, block, 0, s, a);
    return hipGetLastError();
}

template <int DK, int NV>
static hipError_t walk_vec(int vec, bool states, const WalkArgs& a, hipStream_t s) {
    if (vec == 8) return walk_go<DK, NV, 8>(states, a, s);
    return vec == 4 ? walk_go<DK, NV, 4>(states, a, s) : walk_go<DK, NV, 1>(states, a, s);
}

hipError_t launch_walk(const WalkShape& w, bool states_only, const WalkArgs& a, hipStream_t s) {
    int vec = a.k.vec < a.v.vec ? a.k.vec : a.v.vec;
    if (!states_only && a.q.vec < vec) vec = a.q.vec;
    if (w.DK == 64) return w.NV == 32 ? walk_vec<64, 32>(vec, states_only, a, s) : walk_vec<64, 16>(vec, states_only, a, s);
    if (w.DK == 128) return w.NV == 32 ? walk_vec<128, 32>(vec, states_only, a, s) : walk_vec<128, 16>(vec, states_only, a, s);
    return walk_vec<256, 16>(vec, states_only, a, s);
}

hipError_t launch_scan(const ScanArgs& a, hipStream_t s) {
    const dim3 grid(static_cast<uint32_t>(a.nseq * a.HV * (a.floats / 1024)));
    hipLaunchKernelGGL(cconv_linattn_scan_kernel, grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_seg_plan(const int32_t* cu, int64_t nseq, int64_t total, int64_t seg_rows, int32_t* status,
                           int32_t* seq_seg, int32_t* seg_of, int64_t segments, hipStream_t s) {
    hipLaunchKernelGGL(cconv_linattn_plan_kernel, dim3(1), dim3(1024), 0, s, cu, nseq, total, seg_rows, status, seq_seg,
                       seg_of, segments);
    return hipGetLastError();
}

hipError_t launch_group_sum(const GroupSumArgs& a, hipStream_t s) {
    const int64_t blocks = (a.B * a.T * a.H * a.dim + 255) / 256;
    hipLaunchKernelGGL(cconv_linattn_group_sum_kernel, dim3(static_cast<uint32_t>(blocks < 65536 ? blocks : 65536)), dim3(256),
                       0, s, a);
    return hipGetLastError();
}

}  // namespace cconv
