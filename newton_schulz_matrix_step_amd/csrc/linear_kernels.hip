// gfx950 kernels of the linear layer's three products:
//
//   forward          y  = act(x W + b) + residual           (z = x W + b kept, also in 8 bits)
//   input gradient   dx = (dy W^T) act'(z) + add            (act(z) written beside it)
//   weight gradient  dW = x^T dy, db = column sums of dy    (x also from its 8-bit checkpoint)
//
// Each is one product C = A B over k with its own operand layouts and epilogue;
// products run on the matrix cores (v_mfma_f32_16x16x32_bf16, or
// v_mfma_f32_16x16x4_f32 for float32 tensors) with float32 sums, and every
// result is rounded once, at its store.

#include <type_traits>

#include "layer_device.hpp"

namespace muon {
namespace {

using namespace layer;

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short i16x4_t __attribute__((ext_vector_type(4)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));
#ifndef LDS_AS
#define LDS_AS __attribute__((address_space(3)))
#endif

// ---------------------------------------------------------------------------
// global -> LDS
// ---------------------------------------------------------------------------
constexpr uint32_t kFar = 0x80000000u;        // beyond every buffer below: such a lane reads zeros
constexpr uint32_t kMaxRecords = 0x7FFFFFFFu;

__device__ __forceinline__ i32x4_t buffer_at(const char* p, uint32_t bytes) {
    const uint64_t u = reinterpret_cast<uint64_t>(p);
    i32x4_t r;
    r[0] = __builtin_amdgcn_readfirstlane(int(uint32_t(u)));
    r[1] = __builtin_amdgcn_readfirstlane(int(uint32_t(u >> 32) & 0xFFFFu));
    r[2] = __builtin_amdgcn_readfirstlane(int(bytes));
    r[3] = 0x00020000;                        // raw buffer of 32-bit data
    return r;
}

#ifndef MUON_BUFFER_TO_LDS
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// 16 bytes per lane from the buffer straight into LDS: lane L's bytes land at
// lds + 16 L (lds wave-uniform); a lane whose offset lies past the buffer's end
// stores zeros.  Nothing is returned in registers; completion counts in vmcnt.
__device__ __forceinline__ void buffer_to_lds(i32x4_t buf, uint32_t voff, char* lds) {
    const uint32_t a = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(reinterpret_cast<uintptr_t>((LDS_AS char*)lds)));
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(a), "v"(voff), "s"(buf)
                 : "memory", "m0");
}
#pragma clang diagnostic pop
#else
#define buffer_to_lds MUON_BUFFER_TO_LDS
#endif

template <int N>
__device__ __forceinline__ void vm_wait() {   // s_waitcnt vmcnt(N), no wait on the other counters
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

template <class T>
struct Num;
template <>
struct Num<uint16_t> {
    static constexpr int dt = 0, BK = 64, EPC = 8;   // k per stage, elements of a 16-byte chunk
};
template <>
struct Num<float> {
    static constexpr int dt = 1, BK = 32, EPC = 4;
};

// Where an operand comes from: S_DMA whole aligned 16-byte chunks straight into
// LDS; S_ANY any alignment and size, element by element through registers;
// S_ACT8 8-bit codes, decoded on their way through registers.
enum Src { S_DMA, S_ANY, S_ACT8 };

// One stage of one operand is 16 KB of LDS for a 128-wide tile.  Row-contiguous
// operands (KC) lie as [row][8 chunks of 16 bytes along k], chunk XOR row & 7;
// k-strided ones as [k][128 elements] with their own chunk swizzle.  Both feed
// the fragment reads below without bank conflicts.
constexpr int kOpBytes = 16384;

// bf16 [k][128]: a ds_read_b64_tr_b16 group of 16 lanes reads 4 k rows x 32
// bytes (bits 1-2 spread them over a 128-byte window, bit 3 moves the
// neighbouring group to the other half); float32 [k][128]: the four lane groups
// read rows 4 apart, which bits 2-3 put on different 64-byte windows.
template <class T>
__device__ __forceinline__ int ks_swizzle(int k) {
    if constexpr (Num<T>::dt == 0) return ((2 * k) & 6) | ((((k >> 3) ^ (k >> 2)) & 1) << 3);
    else return ((k >> 2) & 3) << 2;
}

// The operand's rows (KC) or columns (KS) [e0, e0 + 128) of the tile, `ext`
// existing in all; k runs to kend.
template <class T, bool KC, int SRC>
struct Loader {
    using N = Num<T>;
    static constexpr int ES = sizeof(T);
    static constexpr int CPR = KC ? 8 : 128 * ES / 16;   // chunks of an LDS row
    static constexpr int RPB = 64 / CPR;                 // LDS rows of 1 KB
    const char* base;
    int64_t ld, ext, kend, e0;
    const uint8_t* exps;
    int64_t lde;
    bool vec8;
    uint32_t voff[4];
    u32x4_t reg[SRC == S_DMA ? 1 : 4];
    int wave, lane;

    // LDS row and logical chunk of this lane's part of 1 KB block q
    __device__ __forceinline__ int lrow(int q) const { return (wave * 4 + q) * RPB + lane / CPR; }
    __device__ __forceinline__ int lchunk(int q) const {
        const int r = lrow(q), c = lane % CPR;
        return KC ? c ^ (r & 7) : c ^ ks_swizzle<T>(r);
    }

    __device__ __forceinline__ void init(const void* p, int64_t ld_, int64_t ext_, int64_t e0_, int64_t kend_, int wave_,
                                         int lane_) {
        ld = ld_;
        ext = ext_;
        e0 = e0_;
        kend = kend_;
        wave = wave_;
        lane = lane_;
        base = static_cast<const char*>(p);
        if constexpr (SRC == S_DMA) {
            base += (KC ? e0 * ld : e0) * ES;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int r = lrow(q), c = lchunk(q);
                const bool in = KC ? e0 + r < ext : e0 + c * N::EPC < ext;
                voff[q] = in ? uint32_t(r * ld * ES + c * 16) : kFar;
            }
        }
    }

    // S_DMA: enqueue the stage at k0 into LDS at st
    __device__ __forceinline__ void issue(int64_t k0, char* st) {
        if constexpr (SRC == S_DMA) {
            if constexpr (KC) {
                const i32x4_t buf = buffer_at(base + k0 * ES, kMaxRecords);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const bool in = k0 + lchunk(q) * N::EPC < kend;   // a whole chunk is in or out
                    buffer_to_lds(buf, in ? voff[q] : kFar, st + (wave * 4 + q) * 1024);
                }
            } else {
                int64_t n = (kend - k0) * ld * ES;   // rows past kend lie past the buffer
                n = n < 0 ? 0 : (n > int64_t(kMaxRecords) ? int64_t(kMaxRecords) : n);
                const i32x4_t buf = buffer_at(base + k0 * ld * ES, uint32_t(n));
#pragma unroll
                for (int q = 0; q < 4; ++q) buffer_to_lds(buf, voff[q], st + (wave * 4 + q) * 1024);
            }
        }
    }

    // S_ANY, S_ACT8: load the stage at k0 into registers
    __device__ __forceinline__ void fetch(int64_t k0) {
        if constexpr (SRC == S_ANY) {
            const GMEM T* p = gm(reinterpret_cast<const T*>(base));
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int64_t r = KC ? e0 + lrow(q) : k0 + lrow(q);
                const int64_t c = (KC ? k0 : e0) + lchunk(q) * N::EPC;
                const int64_t rn = KC ? ext : kend, cn = KC ? kend : ext;
                uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                for (int e = 0; e < N::EPC; ++e) {
                    if (r < rn && c + e < cn) {
                        if constexpr (N::dt == 0) w[e / 2] |= uint32_t(p[r * ld + c + e]) << (16 * (e & 1));
                        else w[e] = __float_as_uint(p[r * ld + c + e]);
                    }
                }
                reg[q] = u32x4_t{w[0], w[1], w[2], w[3]};
            }
        } else if constexpr (SRC == S_ACT8) {
            static_assert(!KC, "checkpoints are stored by rows of k here");
            const GMEM int8_t* p = gm(reinterpret_cast<const int8_t*>(base));
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int64_t k = k0 + lrow(q);
                const int64_t c = e0 + lchunk(q) * N::EPC;
                u32x4_t r = {0u, 0u, 0u, 0u};   // codes in [0..1], the exponent byte in [2]
                if (k < kend && c < ext) {
                    if (vec8 && c + N::EPC <= ext) {
                        if constexpr (N::EPC == 8) {
                            const u32x2_t t = *reinterpret_cast<const GMEM u32x2_t*>(p + k * ld + c);
                            r[0] = t[0];
                            r[1] = t[1];
                        } else {
                            r[0] = *reinterpret_cast<const GMEM uint32_t*>(p + k * ld + c);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < N::EPC; ++e)
                            if (c + e < ext) r[e / 4] |= uint32_t(uint8_t(p[k * ld + c + e])) << (8 * (e & 3));
                    }
                    r[2] = gm(exps)[k * lde + c / kAct8Group];
                }
                reg[q] = r;
            }
        }
    }
    // and store them to LDS.  code * 2^k has at most 7 significant bits, so the
    // bf16 value is its float32 value's upper half, exactly.
    __device__ __forceinline__ void put(char* st) {
        if constexpr (SRC == S_ANY) {
#pragma unroll
            for (int q = 0; q < 4; ++q) *reinterpret_cast<u32x4_t*>(st + (wave * 4 + q) * 1024 + lane * 16) = reg[q];
        } else if constexpr (SRC == S_ACT8) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float step = act8_step(reg[q][2]);
                float v[8];
                act8_dec4(reg[q][0], step, v);
                u32x4_t w;
                if constexpr (N::EPC == 8) {
                    act8_dec4(reg[q][1], step, v + 4);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[e] = (__float_as_uint(v[2 * e]) >> 16) | (__float_as_uint(v[2 * e + 1]) & 0xFFFF0000u);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[e] = __float_as_uint(v[e]);
                }
                *reinterpret_cast<u32x4_t*>(st + (wave * 4 + q) * 1024 + lane * 16) = w;
            }
        }
    }
};

// ---------------------------------------------------------------------------
// LDS -> fragments.  bf16: 8 k values k = 32 s + 8 (lane >> 4) + e of row or
// column rc + (lane & 15).  float32: 4 values k = 16 s + 4 (lane >> 4) + e, one
// for each of four MFMAs; both operands use the same k for the same lane group
// and e, which is all a sum over k asks for.
// ---------------------------------------------------------------------------
template <class T, bool KC>
__device__ __forceinline__ auto frag(const char* lds, int rc, int s, int lane) {
    const int g = lane >> 4, i = lane & 15;
    if constexpr (KC) {
        const int r = rc + i;
        const u32x4_t w = *reinterpret_cast<const u32x4_t*>(lds + r * 128 + (((4 * s + g) ^ (r & 7)) << 4));
        if constexpr (Num<T>::dt == 0) return __builtin_bit_cast(bf16x8_t, w);
        else return __builtin_bit_cast(f32x4_t, w);
    } else if constexpr (Num<T>::dt == 0) {
        const int n = rc + 4 * (i & 3);
        i16x4_t h[2];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            const int k = 32 * s + 8 * g + 4 * hh + (i >> 2);
            const char* p = lds + k * 256 + (((n >> 3) ^ ks_swizzle<T>(k)) << 4) + (n & 7) * 2;
            h[hh] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LDS_AS i16x4_t*)(p));
        }
        return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
        f32x4_t v;
        const int n = rc + i;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int k = 16 * s + 4 * g + e;
            v[e] = *reinterpret_cast<const float*>(lds + k * 512 + (((n >> 2) ^ ks_swizzle<T>(k)) << 4) + (n & 3) * 4);
        }
        return v;
    }
}

__device__ __forceinline__ f32x4_t mma(bf16x8_t a, bf16x8_t b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4_t mma(f32x4_t a, f32x4_t b, f32x4_t c) {
#pragma unroll
    for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
    return c;
}
template <class F>
__device__ __forceinline__ F ones() {
    F f;
    if constexpr (std::is_same_v<F, bf16x8_t>) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = (__bf16)1.f;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = 1.f;
    }
    return f;
}

// ---------------------------------------------------------------------------
// epilogue
// ---------------------------------------------------------------------------
// Two neighbouring 16 x 16 accumulators hold, per lane, 4 consecutive output
// elements of each tile (elements 4 g .. 4 g + 3, g = lane >> 4).  After the two
// swaps lane group g holds the 8 consecutive elements 8 g .. 8 g + 7 of the 32.
__device__ __forceinline__ void join_tiles(f32x4_t a, f32x4_t b, float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        typedef unsigned u2 __attribute__((ext_vector_type(2)));
        const u2 s = __builtin_amdgcn_permlane32_swap(__float_as_uint(a[e]), __float_as_uint(b[e]), false, false);
        const u2 t = __builtin_amdgcn_permlane16_swap(s[0], s[1], false, false);
        v[e] = __uint_as_float(t[0]);
        v[4 + e] = __uint_as_float(t[1]);
    }
}

// 8 consecutive elements (r, c ..) of the output, nv of them inside (0: none).
// SH: lane distance between the four lanes that share a group of 32 columns.
template <int SH>
__device__ __forceinline__ void epilogue8(const LinArgs& a, int64_t r, int64_t c, int nv, float (&v)[8]) {
    const int kind = a.kind;
    if (kind == LIN_FWD) {
        if (a.bias) {
            float b[8];
            load8(a.bias, c, a.bias_dt, false, nv, b);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] += b[k];
        }
        if (a.z && nv > 0) store8(a.z, r * a.ld_z + c, a.dt, a.z_vec, nv, v);
        if (a.z8.codes) {
            float m = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) m = max_mag(m, k < nv ? v[k] : 0.f);
            m = max_mag(m, __shfl_xor(m, SH, 64));
            m = max_mag(m, __shfl_xor(m, 2 * SH, 64));
            if (nv > 0) {
                const uint32_t e = act8_exp(m);
                GMEM int8_t* p = gm(a.z8.codes) + r * a.z8.ld + c;
                if (a.z8.vec && nv >= 8) {
                    u32x2_t w = {0u, 0u};
#pragma unroll
                    for (int k = 0; k < 8; ++k) w[k >> 2] |= act8_code(v[k], e) << (8 * (k & 3));
                    *reinterpret_cast<GMEM u32x2_t*>(p) = w;
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (k < nv) p[k] = int8_t(act8_code(v[k], e));
                }
                if ((c & (kAct8Group - 1)) == 0) gm(a.z8.exps)[r * a.z8.lde + c / kAct8Group] = uint8_t(e);
            }
        }
        if (nv <= 0) return;
        if (a.act != ACT_NONE) {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = act_value(v[k], a.act);
        }
    } else if (kind == LIN_DX) {
        if (nv <= 0) return;
        if (a.z || a.z8.codes) {
            float z[8], h[8];
            if (a.z) {
                load8(a.z, r * a.ld_z + c, a.dt, a.z_vec, nv, z);
            } else {
                const float step = act8_step(gm(a.z8.exps)[r * a.z8.lde + c / kAct8Group]);
                const GMEM int8_t* p = gm(a.z8.codes) + r * a.z8.ld + c;
                if (a.z8.vec && nv >= 8) {
                    const u32x2_t w = *reinterpret_cast<const GMEM u32x2_t*>(p);
                    act8_dec4(w[0], step, z);
                    act8_dec4(w[1], step, z + 4);
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) z[k] = k < nv ? float(p[k]) * step : 0.f;
                }
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                float d;
                act_both(z[k], a.act, h[k], d);
                v[k] *= d;
            }
            if (a.act_out) store8(a.act_out, r * a.ld_act + c, a.dt, a.act_vec, nv, h);
        }
    } else {
        if (nv <= 0) return;
        if (a.accumulate) {
            float o[8];
            load8(a.out, r * a.ld_out + c, a.out_dt, a.out_vec, nv, o);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] += o[k];
        }
    }
    if (a.add) {
        float b[8];
        load8(a.add, r * a.ld_add + c, a.dt, a.add_vec, nv, b);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += b[k];
    }
    store8(a.out, r * a.ld_out + c, a.out_dt, a.out_vec, nv, v);
}

// Shape of the output as stored, and of the split sums (rows padded to whole groups).
struct OutShape {
    int64_t rows, cols, ldp;
};
__host__ __device__ inline OutShape out_shape(const LinArgs& a) {
    OutShape o;
    o.rows = a.out_trans ? a.N : a.M;
    o.cols = a.out_trans ? a.M : a.N;
    o.ldp = (o.cols + kAct8Group - 1) / kAct8Group * kAct8Group;
    return o;
}

// 8 elements of this workgroup's tile: straight to the result, or to the sums
// of its split.
__device__ __forceinline__ void emit8(const LinArgs& a, const OutShape& o, int split, int64_t r, int64_t c,
                                      float (&v)[8]) {
    int64_t n = o.cols - c;
    n = r < o.rows ? (n > 8 ? 8 : n) : 0;
    if (a.splits > 1) {
        if (n > 0) {   // the row's padding takes whole runs
            GMEM float* p = gm(a.partial) + (int64_t(split) * o.rows + r) * o.ldp + c;
            *reinterpret_cast<GMEM f32x4_t*>(p) = f32x4_t{v[0], v[1], v[2], v[3]};
            *reinterpret_cast<GMEM f32x4_t*>(p + 4) = f32x4_t{v[4], v[5], v[6], v[7]};
        }
        return;
    }
    epilogue8<16>(a, r, c, n > 0 ? int(n) : 0, v);
}

__device__ __forceinline__ void emit_db(const LinArgs& a, int split, int64_t n, float v) {
    if (n >= a.N) return;
    if (a.splits > 1) {
        gm(a.db_partial)[int64_t(split) * a.N + n] = v;
        return;
    }
    if (a.accumulate) v += load1(a.db, n, a.db_dt);
    store1(a.db, n, a.db_dt, v);
}

// Workgroup -> (split, tile).  Workgroup b runs on XCD b % 8 and each XCD has
// its own L2: an XCD takes one contiguous eighth of the tiles, in groups of 8
// tile rows across all tile columns, so that the tiles it runs at one time
// share few operand panels.
struct TileAt {
    int64_t tm, tn;
    int split;
    bool in;
};
__device__ __forceinline__ TileAt tile_at(const LinArgs& a, int edge) {
    const int64_t nm = (a.M + edge - 1) / edge, nn = (a.N + edge - 1) / edge, all = nm * nn * a.splits;
    const int64_t chunk = (all + 7) / 8;
    const int64_t t = int64_t(blockIdx.x & 7) * chunk + (blockIdx.x >> 3);
    TileAt o;
    o.in = t < all && int64_t(blockIdx.x >> 3) < chunk;
    o.split = int(t / (nm * nn));
    const int64_t u = t % (nm * nn), g = u / (8 * nn), rows = nm - 8 * g < 8 ? nm - 8 * g : 8, w = u % (8 * nn);
    o.tm = 8 * g + w % rows;
    o.tn = w / rows;
    return o;
}

// ---------------------------------------------------------------------------
// 128 x 128 tiles: 4 waves of 64 x 64, two LDS stages (64 KB, so two workgroups
// share a CU and one's epilogue overlaps the other's main loop).
// TR: the accumulators hold runs along M (the output is stored transposed).
// ---------------------------------------------------------------------------
template <class T, bool AKC, bool BKC, int ASRC, int BSRC, bool TR>
__global__ __launch_bounds__(256) void linear_tile_kernel(LinArgs a) {
    using N = Num<T>;
    __shared__ __align__(1024) char smem[4 * kOpBytes];
    const TileAt t = tile_at(a, 128);
    if (!t.in) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const int64_t nkb = (a.K + N::BK - 1) / N::BK, kbs = (nkb + a.splits - 1) / a.splits;
    const int64_t kb0 = t.split * kbs, kb1 = kb0 + kbs < nkb ? kb0 + kbs : nkb;
    const int64_t kend = kb1 * N::BK < a.K ? kb1 * N::BK : a.K;
    Loader<T, AKC, ASRC> la;
    Loader<T, BKC, BSRC> lb;
    la.init(a.a, a.lda, a.M, t.tm * 128, kend, wave, lane);
    lb.init(a.b, a.ldb, a.N, t.tn * 128, kend, wave, lane);
    if constexpr (ASRC == S_ACT8) {
        la.exps = a.a_exps;
        la.lde = a.lda_exps;
        la.vec8 = a.a8_vec != 0;
    }
    const int wr = (wave >> 1) * 64, wc = (wave & 1) * 64;
    f32x4_t acc[4][4];
    f32x4_t dbs[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        dbs[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    // the column sums of B: a product with a row of ones, in the tiles of the first tile row
    const bool sum_b = a.db != nullptr && t.tm == 0 && wr == 0;

    if (kb0 < kb1) {
        la.issue(kb0 * N::BK, smem);
        lb.issue(kb0 * N::BK, smem + kOpBytes);
        la.fetch(kb0 * N::BK);
        lb.fetch(kb0 * N::BK);
        la.put(smem);
        lb.put(smem + kOpBytes);
    }
    for (int64_t kb = kb0; kb < kb1; ++kb) {
        char* cur = smem + ((kb - kb0) & 1) * 2 * kOpBytes;
        char* nxt = smem + ((kb - kb0 + 1) & 1) * 2 * kOpBytes;
        vm_wait<0>();        // this wave's part of the stage has landed
        __syncthreads();     // and every other wave's; the other stage is free
        const bool more = kb + 1 < kb1;
        if (more) {
            la.issue((kb + 1) * N::BK, nxt);
            lb.issue((kb + 1) * N::BK, nxt + kOpBytes);
            la.fetch((kb + 1) * N::BK);
            lb.fetch((kb + 1) * N::BK);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            decltype(frag<T, AKC>(cur, 0, 0, 0)) fa[4], fb[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) fa[i] = frag<T, AKC>(cur, wr + 16 * i, s, lane);
#pragma unroll
            for (int j = 0; j < 4; ++j) fb[j] = frag<T, BKC>(cur + kOpBytes, wc + 16 * j, s, lane);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = TR ? mma(fa[i], fb[j], acc[i][j]) : mma(fb[j], fa[i], acc[i][j]);
            if (sum_b) {
                const auto one = ones<decltype(frag<T, BKC>(cur, 0, 0, 0))>();
#pragma unroll
                for (int j = 0; j < 4; ++j) dbs[j] = mma(fb[j], one, dbs[j]);
            }
        }
        if (more) {
            la.put(nxt);
            lb.put(nxt + kOpBytes);
        }
    }

    const OutShape o = out_shape(a);
    const int64_t m0 = t.tm * 128 + wr, n0 = t.tn * 128 + wc;
    const int g = lane >> 4, i16 = lane & 15;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            float v[8];
            if constexpr (TR) {   // column n0 + 16 i + i16 of C, rows m0 + 32 p + 8 g ..
                join_tiles(acc[2 * p][i], acc[2 * p + 1][i], v);
                emit8(a, o, t.split, n0 + 16 * i + i16, m0 + 32 * p + 8 * g, v);
            } else {
                join_tiles(acc[i][2 * p], acc[i][2 * p + 1], v);
                emit8(a, o, t.split, m0 + 16 * i + i16, n0 + 32 * p + 8 * g, v);
            }
        }
    if (sum_b && i16 == 0) {   // every column of the product with ones is the same
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) emit_db(a, t.split, n0 + 16 * j + 4 * g + e, dbs[j][e]);
    }
}

// ---------------------------------------------------------------------------
// The splits' sums, added in order, through the epilogue: 8 elements a lane.
// The workgroups past the output's join the column sums.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void linear_join_kernel(LinArgs a, int64_t out_blocks) {
    if (int64_t(blockIdx.x) >= out_blocks) {
        const int64_t n = (int64_t(blockIdx.x) - out_blocks) * 256 + threadIdx.x;
        if (n >= a.N) return;
        float v = 0.f;
        for (int s = 0; s < a.splits; ++s) v += gm(a.db_partial)[int64_t(s) * a.N + n];
        if (a.accumulate) v += load1(a.db, n, a.db_dt);
        store1(a.db, n, a.db_dt, v);
        return;
    }
    const OutShape o = out_shape(a);
    const int64_t rpr = o.ldp / 8;                       // runs per row, a multiple of 4
    const int64_t idx = int64_t(blockIdx.x) * 256 + threadIdx.x;
    const int64_t r = idx / rpr, c = (idx % rpr) * 8;
    int64_t n = o.cols - c;
    n = r < o.rows ? (n > 8 ? 8 : n) : 0;
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = 0.f;
    if (n > 0) {
        const GMEM float* p = gm(a.partial) + r * o.ldp + c;
        for (int s = 0; s < a.splits; ++s, p += o.rows * o.ldp) {
            const f32x4_t x = *reinterpret_cast<const GMEM f32x4_t*>(p);
            const f32x4_t y = *reinterpret_cast<const GMEM f32x4_t*>(p + 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[k] += x[k];
                v[4 + k] += y[k];
            }
        }
    }
    epilogue8<1>(a, r, c, n > 0 ? int(n) : 0, v);
}

template <class T, bool AKC, bool BKC, int ASRC, int BSRC, bool TR>
hipError_t launch_tile(const LinArgs& a, hipStream_t s) {
    const int64_t nm = (a.M + 127) / 128, nn = (a.N + 127) / 128, all = nm * nn * a.splits;
    hipLaunchKernelGGL((linear_tile_kernel<T, AKC, BKC, ASRC, BSRC, TR>), dim3(unsigned((all + 7) / 8 * 8)), dim3(256),
                       0, s, a);
    return hipGetLastError();
}

template <class T>
hipError_t launch_typed(const LinArgs& a, hipStream_t s) {
    // element-wise loads for both operands where either needs them
    const bool dma = a.a_dma && a.b_dma;
    if (a.kind != LIN_DW) {
        if (a.b_kc)
            return dma ? launch_tile<T, true, true, S_DMA, S_DMA, false>(a, s)
                       : launch_tile<T, true, true, S_ANY, S_ANY, false>(a, s);
        return dma ? launch_tile<T, true, false, S_DMA, S_DMA, false>(a, s)
                   : launch_tile<T, true, false, S_ANY, S_ANY, false>(a, s);
    }
    if (a.a_exps) {
        if (a.out_trans)
            return a.b_dma ? launch_tile<T, false, false, S_ACT8, S_DMA, true>(a, s)
                           : launch_tile<T, false, false, S_ACT8, S_ANY, true>(a, s);
        return a.b_dma ? launch_tile<T, false, false, S_ACT8, S_DMA, false>(a, s)
                       : launch_tile<T, false, false, S_ACT8, S_ANY, false>(a, s);
    }
    if (a.out_trans)
        return dma ? launch_tile<T, false, false, S_DMA, S_DMA, true>(a, s)
                   : launch_tile<T, false, false, S_ANY, S_ANY, true>(a, s);
    return dma ? launch_tile<T, false, false, S_DMA, S_DMA, false>(a, s)
               : launch_tile<T, false, false, S_ANY, S_ANY, false>(a, s);
}

}  // namespace

LinPlan plan_linear(const LinArgs& a) {
    LinPlan p;
    p.tile = 128;
    const int64_t tiles = ((a.M + 127) / 128) * ((a.N + 127) / 128);
    const int64_t bk = a.dt == 0 ? 64 : 32, nkb = (a.K + bk - 1) / bk;
    // two workgroups a CU; a split keeps at least 4 k blocks
    int64_t s = 1;
    if (tiles < 512) {
        s = 512 / tiles;
        s = s < nkb / 4 ? s : nkb / 4;
        s = s < 1 ? 1 : (s > 64 ? 64 : s);
        if (s > 1) {   // no empty split
            const int64_t per = (nkb + s - 1) / s;
            s = (nkb + per - 1) / per;
        }
    }
    p.splits = int(s);
    if (s > 1) {
        const OutShape o = out_shape(a);
        p.partial_bytes = size_t(s) * size_t(o.rows) * size_t(o.ldp) * 4;
        p.db_bytes = a.db ? size_t(s) * size_t(a.N) * 4 : 0;
    }
    return p;
}

hipError_t launch_linear(const LinArgs& a, hipStream_t s) {
    if (a.M <= 0 || a.N <= 0) return hipSuccess;
    hipError_t e = a.dt == 0 ? launch_typed<uint16_t>(a, s) : launch_typed<float>(a, s);
    if (e != hipSuccess || a.splits <= 1) return e;
    const OutShape o = out_shape(a);
    const int64_t ob = (o.rows * (o.ldp / 8) + 255) / 256, db = a.db ? (a.N + 255) / 256 : 0;
    hipLaunchKernelGGL(linear_join_kernel, dim3(unsigned(ob + db)), dim3(256), 0, s, a, ob);
    return hipGetLastError();
}

}  // namespace muon
