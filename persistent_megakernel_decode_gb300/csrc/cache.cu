// 8-bit paged KV cache: storing tokens (quantisation), loading them back,
// copying pages.  All three are bound by memory: store reads 2 bytes and
// writes 1 per element, load the reverse, copy reads and writes 1.  Measured
// (one GB300, device time; a plain copy reaches 6.8 TB/s): 8 contexts of
// 512-4096 tokens of the 1B shape stored in 132 us (6.8 TB/s), 4 x 2048 tokens
// of the 8B shape loaded in 265 us (6.8 TB/s), 300 pages of the 8B shape copied
// in 410 us (6.9 TB/s, the plain copy's rate within 2 %).
#include "dev_serve.cuh"

#include <algorithm>
#include <cstring>
#include <new>
#include <vector>

namespace mk {

int cache_check(const mk_cache_desc *c, CacheView &v) {
    if (!c) return set_error(MK_ERR_INVALID, "null cache descriptor");
    if (c->layers <= 0 || c->pages <= 0 || c->kv_heads <= 0)
        return set_error(MK_ERR_INVALID, "layers, pages and kv_heads must be positive");
    if (c->page_tokens != 32 && c->page_tokens != 64)
        return set_error(MK_ERR_UNSUPPORTED, "page_tokens must be 32 or 64");
    if (c->head_dim != 64 && c->head_dim != 128) return set_error(MK_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
    if (!c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales || !c->status)
        return set_error(MK_ERR_INVALID, "null cache buffer");
    if ((c->k_codes | c->v_codes) % 16 || (c->k_scales | c->v_scales | c->status) % 4)
        return set_error(MK_ERR_INVALID, "cache codes must be 16-byte aligned, scales and status 4-byte");
    if (c->kv_heads > 65535 || c->layers > 65535) return set_error(MK_ERR_UNSUPPORTED, "too many layers or kv heads");
    v.k = reinterpret_cast<uint8_t *>(c->k_codes);
    v.v = reinterpret_cast<uint8_t *>(c->v_codes);
    v.ks = reinterpret_cast<float *>(c->k_scales);
    v.vs = reinterpret_cast<float *>(c->v_scales);
    v.status = reinterpret_cast<int *>(c->status);
    v.layers = c->layers;
    v.pages = c->pages;
    v.hkv = c->kv_heads;
    return MK_OK;
}

struct RowsView {
    uint16_t *k, *v;
    int64_t ks[4], vs[4];
    int rows;
    const int *row0;
};

struct MoveParams {
    CacheView c;
    RowsView r;
    const int *table, *start, *count;
    int width, max_count;
};

// The tokens [lo, hi) of sequence b on its slot-th touched page, and that
// page's number as the table has it (page_ok checks it: what does not need the
// page may load meanwhile); false if there are none or a check fails.
template <int P>
DEV bool page_span(const MoveParams &m, int b, int slot, int &first, int &lo, int &hi, int &page, int &src0) {
    const int s = m.start[b], n = m.count[b];
    const int r0 = m.r.row0 ? m.r.row0[b] : 0;
    if (n == 0) return false;
    const bool reports = slot == 0 && threadIdx.x % 32 == 0;
    if (s < 0 || n < 0 || n > m.max_count || r0 < 0 || r0 > m.r.rows || n > m.r.rows - r0 ||
        (int64_t)s + n > (int64_t)m.width * P) {
        if (reports) note_failure(m.c.status, MK_ERR_DEVICE_CHECK, b, s, -1);
        return false;
    }
    const int j = s / P + slot;
    if ((int64_t)j * P >= (int64_t)s + n) return false;
    first = j * P;
    lo = max(s, first);
    hi = first + min(s - first + n, P);
    src0 = r0 - s;
    page = __ldg(&m.table[(size_t)b * m.width + j]);
    return true;
}
DEV bool page_ok(const MoveParams &m, int b, int first, int page) {
    if ((unsigned)page < (unsigned)m.c.pages) return true;
    if (threadIdx.x % 32 == 0) note_failure(m.c.status, MK_ERR_DEVICE_CHECK, b, first, page);
    return false;
}

// Largest finite magnitude of 8 bf16 values, as bf16 bits (they order like
// integers without their sign).
DEV uint32_t amax8(uint4 x) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w;
        const uint32_t lo = w & 0x7fffu, hi = (w >> 16) & 0x7fffu;
        m = max(m, lo < 0x7f80u ? lo : 0u);
        m = max(m, hi < 0x7f80u ? hi : 0u);
    }
    return m;
}

// The least power of two s with amax / s <= 448 = 1.75 x 2^8, held to 2^-120
// .. 2^120 (0 for amax 0); amax as bf16 bits: exponent in the upper 8, 96 of
// 128 fraction steps is 1.75.
DEV float page_scale(uint32_t a) {
    if (a == 0) return 0.f;
    const int e = min(max((int)(a >> 7) - 127 - 8 + ((a & 0x7fu) > 96u ? 1 : 0), -120), 120);
    return __uint_as_float((uint32_t)(e + 127) << 23);
}
// 1 / s of such a scale, exact (1 for 0).
DEV float page_inverse(float s) { return s > 0.f ? __uint_as_float((254u << 23) - __float_as_uint(s)) : 1.f; }

DEV uint2 encode8(uint4 x, float inv) {
    uint2 r;
    r.x = to_e4m3x2(__uint_as_float(x.x << 16) * inv, __uint_as_float(x.x & 0xffff0000u) * inv) |
          (to_e4m3x2(__uint_as_float(x.y << 16) * inv, __uint_as_float(x.y & 0xffff0000u) * inv) << 16);
    r.y = to_e4m3x2(__uint_as_float(x.z << 16) * inv, __uint_as_float(x.z & 0xffff0000u) * inv) |
          (to_e4m3x2(__uint_as_float(x.w << 16) * inv, __uint_as_float(x.w & 0xffff0000u) * inv) << 16);
    return r;
}

// 4 x 4 bytes transposed: word i of the result holds byte i of a, b, c, d.
DEV void transpose4(uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t (&o)[4]) {
    const uint32_t ab0 = __byte_perm(a, b, 0x5140), ab1 = __byte_perm(a, b, 0x7362);
    const uint32_t cd0 = __byte_perm(c, d, 0x5140), cd1 = __byte_perm(c, d, 0x7362);
    o[0] = __byte_perm(ab0, cd0, 0x5410);
    o[1] = __byte_perm(ab0, cd0, 0x7632);
    o[2] = __byte_perm(ab1, cd1, 0x5410);
    o[3] = __byte_perm(ab1, cd1, 0x7632);
}

// Codes of a page, rounded to a scale 1 / ratio times as large (ratio a power
// of two: the product is exact in f16 wherever it is not far below e4m3's
// least step, so each code is rounded once).
DEV void rescale_page(uint32_t *w, int words, float ratio, int tid, int threads) {
    const float r = fmaxf(ratio, 0x1p-24f);  // below, every product rounds to 0 as with this
    uint32_t r2;
    asm("cvt.rn.f16x2.f32 %0, %1, %1;" : "=r"(r2) : "f"(r));
    for (int i = tid; i < words; i += threads) {
        const uint32_t x = w[i];
        w[i] = half2_to_e4m3x2(half2_mul(e4m3x2_to_half2(x), r2)) |
               (half2_to_e4m3x2(half2_mul(e4m3x2_to_half2(x >> 16), r2)) << 16);
    }
}

constexpr int MOVE_THREADS = 128;

// One CTA per (touched page, kv head, sequence, layer).  The page's new rows
// are loaded once into registers (K as [token][8 dims], V as 4 tokens x 8
// dims, which transposes in registers: the V codes are written as words of 4
// tokens without a pass through shared memory), the block's two maxima give
// the scales, and the codes are written.
template <int D, int P>
__global__ void __launch_bounds__(MOVE_THREADS) cache_store_kernel(const MoveParams m) {
    constexpr int KV = P * D / 8, KN = KV / MOVE_THREADS;          // K vectors of 8 dims, per thread
    constexpr int VU = (P / 4) * (D / 8), VN = (VU + MOVE_THREADS - 1) / MOVE_THREADS;  // V units of 4 tokens x 8 dims
    __shared__ uint32_t s_max[2][MOVE_THREADS / 32];
    const int h = blockIdx.x % m.c.hkv, slot = blockIdx.x / m.c.hkv, b = blockIdx.y, l = blockIdx.z, tid = threadIdx.x;
    int first, lo, hi, page, src0;
    if (!page_span<P>(m, b, slot, first, lo, hi, page, src0)) return;
    const uint16_t *ksrc = m.r.k + l * m.r.ks[0] + b * m.r.ks[1] + h * m.r.ks[3];
    const uint16_t *vsrc = m.r.v + l * m.r.vs[0] + b * m.r.vs[1] + h * m.r.vs[3];
    uint4 kx[KN], vx[VN][4];
    uint32_t ka = 0, va = 0;
#pragma unroll
    for (int i = 0; i < KN; ++i) {
        const int u = tid + i * MOVE_THREADS, t = first + u / (D / 8);
        kx[i] = make_uint4(0, 0, 0, 0);
        if (t >= lo && t < hi)
            kx[i] = __ldg(reinterpret_cast<const uint4 *>(ksrc + (int64_t)(src0 + t) * m.r.ks[2]) + u % (D / 8));
    }
#pragma unroll
    for (int i = 0; i < VN; ++i) {
        const int u = tid + i * MOVE_THREADS, c = u / (P / 4), t0 = first + (u % (P / 4)) * 4;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            vx[i][j] = make_uint4(0, 0, 0, 0);
            if (u < VU && t0 + j >= lo && t0 + j < hi)
                vx[i][j] = __ldg(reinterpret_cast<const uint4 *>(vsrc + (int64_t)(src0 + t0 + j) * m.r.vs[2]) + c);
        }
    }
    if (!page_ok(m, b, first, page)) return;
    const size_t at = m.c.at(l, page, h);
    uint8_t *kp = m.c.k + at * (P * D), *vp = m.c.v + at * (P * D);
    const bool held = first < lo;
    const float old_k = held ? m.c.ks[at] : 0.f, old_v = held ? m.c.vs[at] : 0.f;
#pragma unroll
    for (int i = 0; i < KN; ++i) ka = max(ka, amax8(kx[i]));
#pragma unroll
    for (int i = 0; i < VN; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) va = max(va, amax8(vx[i][j]));
    ka = __reduce_max_sync(FULL, ka);
    va = __reduce_max_sync(FULL, va);
    if (tid % 32 == 0) {
        s_max[0][tid / 32] = ka;
        s_max[1][tid / 32] = va;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MOVE_THREADS / 32; ++i) {
        ka = max(ka, s_max[0][i]);
        va = max(va, s_max[1][i]);
    }
    const float sk = fmaxf(page_scale(ka), old_k), sv = fmaxf(page_scale(va), old_v);
    if (held && (sk > old_k || sv > old_v)) {
        if (sk > old_k) rescale_page(reinterpret_cast<uint32_t *>(kp), P * D / 4, old_k * page_inverse(sk), tid, MOVE_THREADS);
        if (sv > old_v) rescale_page(reinterpret_cast<uint32_t *>(vp), P * D / 4, old_v * page_inverse(sv), tid, MOVE_THREADS);
        __syncthreads();
    }
    const float ik = page_inverse(sk), iv = page_inverse(sv);
#pragma unroll
    for (int i = 0; i < KN; ++i) {
        const int u = tid + i * MOVE_THREADS, t = first + u / (D / 8);
        if (!held || (t >= lo && t < hi)) reinterpret_cast<uint2 *>(kp)[u] = encode8(kx[i], ik);
    }
#pragma unroll
    for (int i = 0; i < VN; ++i) {
        const int u = tid + i * MOVE_THREADS, c = u / (P / 4), q = u % (P / 4), t0 = first + q * 4;
        if (u >= VU || (held && (t0 + 4 <= lo || t0 >= hi))) continue;
        uint2 e[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) e[j] = encode8(vx[i][j], iv);
        uint32_t w[8], x[4];
        transpose4(e[0].x, e[1].x, e[2].x, e[3].x, x);
        w[0] = x[0], w[1] = x[1], w[2] = x[2], w[3] = x[3];
        transpose4(e[0].y, e[1].y, e[2].y, e[3].y, x);
        w[4] = x[0], w[5] = x[1], w[6] = x[2], w[7] = x[3];
        uint8_t *dst = vp + (size_t)c * 8 * P + q * 4;
        if (!held || (t0 >= lo && t0 + 4 <= hi)) {
#pragma unroll
            for (int d = 0; d < 8; ++d) *reinterpret_cast<uint32_t *>(dst + d * P) = w[d];
        } else {  // a group that also holds earlier tokens (or slots behind the last one)
#pragma unroll
            for (int d = 0; d < 8; ++d)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (t0 + j >= lo && t0 + j < hi) dst[d * P + j] = (uint8_t)(w[d] >> (8 * j));
        }
    }
    if (tid == 0) {
        m.c.ks[at] = sk;
        m.c.vs[at] = sv;
    }
}

// Appending a few tokens (a decode step: one): one warp per (kv head,
// sequence, layer), the lower lanes on K's vectors of 8 dims, the upper on
// V's.  The block form above takes a CTA for each, most of whose threads have
// nothing to do.  16 sequences, 36 layers, 8 heads of 128, this form / the
// block form: 1 token 8.0 / 32 us, 2 13.8 / 37, 4 27.6 / 41, 8 50 / 47, 16 89 /
// 49 (8 sequences, 16 layers, heads of 64: 3.7 / 6.2, 4.1 / 7.0, 6.0 / 7.5, 10.6
// / 8.3, 14.8 / 8.3).  A token's V is one byte in each of D sectors of its page.
constexpr int APPEND_TOKENS = 4;
template <int D, int P>
__global__ void __launch_bounds__(MOVE_THREADS) cache_append_kernel(const MoveParams m, int heads) {
    constexpr int VEC = D / 8;
    const int lane = threadIdx.x % 32;
    const int64_t w = (int64_t)blockIdx.x * (MOVE_THREADS / 32) + threadIdx.x / 32;
    if (w >= (int64_t)heads * m.c.layers) return;  // heads: batch x kv heads
    const int l = (int)(w / heads), bh = (int)(w % heads), b = bh / m.c.hkv, h = bh % m.c.hkv;
    const bool is_v = lane >= VEC, busy = lane < 2 * VEC;
    const int c = lane % VEC;
    const int64_t *st = is_v ? m.r.vs : m.r.ks;
    const uint16_t *src = (is_v ? m.r.v : m.r.k) + l * st[0] + b * st[1] + h * st[3];
    for (int slot = 0; slot < 2; ++slot) {  // at most 4 tokens lie on at most two pages
        int first, lo, hi, page, src0;
        if (!page_span<P>(m, b, slot, first, lo, hi, page, src0)) continue;
        uint4 x[APPEND_TOKENS];
        uint32_t a = 0;
#pragma unroll
        for (int j = 0; j < APPEND_TOKENS; ++j) {
            x[j] = make_uint4(0, 0, 0, 0);
            if (busy && lo + j < hi) x[j] = __ldg(reinterpret_cast<const uint4 *>(src + (int64_t)(src0 + lo + j) * st[2]) + c);
        }
        if (!page_ok(m, b, first, page)) continue;
        const size_t at = m.c.at(l, page, h);
        uint8_t *dst = (is_v ? m.c.v : m.c.k) + at * (P * D);
        float *scale = (is_v ? m.c.vs : m.c.ks) + at;
        const bool held = first < lo;
        const float old = held ? *scale : 0.f;
#pragma unroll
        for (int j = 0; j < APPEND_TOKENS; ++j) a = max(a, amax8(x[j]));
#pragma unroll
        for (int o = 1; o < VEC; o <<= 1) a = max(a, __shfl_xor_sync(FULL, a, o));
        const float s = fmaxf(page_scale(a), old);
        // the whole page, for either half, by all lanes
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const float ns = __shfl_sync(FULL, s, half * VEC), os = __shfl_sync(FULL, old, half * VEC);
            uint8_t *pg = (half ? m.c.v : m.c.k) + at * (P * D);
            if (!held) {
                for (int i = lane; i < P * D / 16; i += 32) reinterpret_cast<uint4 *>(pg)[i] = make_uint4(0, 0, 0, 0);
            } else if (ns > os) {
                rescale_page(reinterpret_cast<uint32_t *>(pg), P * D / 4, os * page_inverse(ns), lane, 32);
            }
        }
        __syncwarp();
        const float inv = page_inverse(s);
        if (busy) {
#pragma unroll
            for (int j = 0; j < APPEND_TOKENS; ++j) {
                if (lo + j >= hi) break;
                const uint2 e = encode8(x[j], inv);
                const int t = lo + j - first;
                if (!is_v) {
                    reinterpret_cast<uint2 *>(dst + t * D)[c] = e;
                } else {
#pragma unroll
                    for (int d = 0; d < 8; ++d) dst[(c * 8 + d) * P + t] = (uint8_t)((d < 4 ? e.x : e.y) >> (8 * (d % 4)));
                }
            }
            if (c == 0) *scale = s;
        }
    }
}

// bf16 values of 8 codes; the product with a power of two is exact (bf16 has
// e4m3's bits and more) short of bf16's own range.
DEV uint4 decode8(uint32_t a, uint32_t b, float s) {
    float f[8];
    half2_floats(e4m3x2_to_half2(a), f[0], f[1]);
    half2_floats(e4m3x2_to_half2(a >> 16), f[2], f[3]);
    half2_floats(e4m3x2_to_half2(b), f[4], f[5]);
    half2_floats(e4m3x2_to_half2(b >> 16), f[6], f[7]);
    return make_uint4(bf16_pair(f[0] * s, f[1] * s), bf16_pair(f[2] * s, f[3] * s), bf16_pair(f[4] * s, f[5] * s),
                      bf16_pair(f[6] * s, f[7] * s));
}

// The inverse of cache_store_kernel, the same split and the same transpose.
template <int D, int P>
__global__ void __launch_bounds__(MOVE_THREADS) cache_load_kernel(const MoveParams m) {
    constexpr int KV = P * D / 8, KN = KV / MOVE_THREADS;
    constexpr int VU = (P / 4) * (D / 8), VN = (VU + MOVE_THREADS - 1) / MOVE_THREADS;
    const int h = blockIdx.x % m.c.hkv, slot = blockIdx.x / m.c.hkv, b = blockIdx.y, l = blockIdx.z, tid = threadIdx.x;
    int first, lo, hi, page, src0;
    if (!page_span<P>(m, b, slot, first, lo, hi, page, src0) || !page_ok(m, b, first, page)) return;
    const size_t at = m.c.at(l, page, h);
    const uint8_t *kp = m.c.k + at * (P * D), *vp = m.c.v + at * (P * D);
    const float sk = m.c.ks[at], sv = m.c.vs[at];
    uint16_t *kdst = m.r.k + l * m.r.ks[0] + b * m.r.ks[1] + h * m.r.ks[3];
    uint16_t *vdst = m.r.v + l * m.r.vs[0] + b * m.r.vs[1] + h * m.r.vs[3];
    uint2 kx[KN];
    uint32_t vx[VN][8];
#pragma unroll
    for (int i = 0; i < KN; ++i) kx[i] = __ldg(reinterpret_cast<const uint2 *>(kp) + tid + i * MOVE_THREADS);
#pragma unroll
    for (int i = 0; i < VN; ++i) {
        const int u = tid + i * MOVE_THREADS, c = u / (P / 4), q = u % (P / 4);
        if (u < VU)
#pragma unroll
            for (int d = 0; d < 8; ++d) vx[i][d] = __ldg(reinterpret_cast<const uint32_t *>(vp + (size_t)(c * 8 + d) * P) + q);
    }
#pragma unroll
    for (int i = 0; i < KN; ++i) {
        const int u = tid + i * MOVE_THREADS, t = first + u / (D / 8);
        if (t >= lo && t < hi)
            reinterpret_cast<uint4 *>(kdst + (int64_t)(src0 + t) * m.r.ks[2])[u % (D / 8)] = decode8(kx[i].x, kx[i].y, sk);
    }
#pragma unroll
    for (int i = 0; i < VN; ++i) {
        const int u = tid + i * MOVE_THREADS, c = u / (P / 4), t0 = first + (u % (P / 4)) * 4;
        if (u >= VU) continue;
        uint32_t a[4], e[4];
        transpose4(vx[i][0], vx[i][1], vx[i][2], vx[i][3], a);
        transpose4(vx[i][4], vx[i][5], vx[i][6], vx[i][7], e);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (t0 + j >= lo && t0 + j < hi)
                reinterpret_cast<uint4 *>(vdst + (int64_t)(src0 + t0 + j) * m.r.vs[2])[c] = decode8(a[j], e[j], sv);
    }
}

// Page pairs travel in the kernel's parameters: no host-to-device copy, and a
// captured launch keeps them.
constexpr int COPY_PAIRS = 480, COPY_THREADS = 256;
struct CopyParams {
    CacheView c;
    int page_bytes, n;
    int *table;
    int64_t entries;
    int src[COPY_PAIRS], dst[COPY_PAIRS];  // by rising src
};

// CTA (i, 2 l + half): half 0 / 1 = K / V of pair i, layer l; the last y row
// renames the table's entries.
__global__ void __launch_bounds__(COPY_THREADS) cache_copy_kernel(const __grid_constant__ CopyParams p) {
    const int tid = threadIdx.x, l = blockIdx.y / 2, i = blockIdx.x;
    if (l == p.c.layers) {
        __shared__ int s_src[COPY_PAIRS], s_dst[COPY_PAIRS];
        for (int k = tid; k < p.n; k += COPY_THREADS) {
            s_src[k] = p.src[k];
            s_dst[k] = p.dst[k];
        }
        __syncthreads();
        for (int64_t e = (int64_t)i * COPY_THREADS + tid; e < p.entries; e += (int64_t)gridDim.x * COPY_THREADS) {
            const int x = p.table[e];
            int a = 0, z = p.n;  // the first src >= x
            while (a < z) {
                const int mid = (a + z) / 2;
                if (s_src[mid] < x) a = mid + 1;
                else z = mid;
            }
            if (a < p.n && s_src[a] == x) p.table[e] = s_dst[a];
        }
        return;
    }
    uint8_t *codes = blockIdx.y & 1 ? p.c.v : p.c.k;
    float *scales = blockIdx.y & 1 ? p.c.vs : p.c.ks;
    const size_t s = (size_t)l * p.c.pages + p.src[i], d = (size_t)l * p.c.pages + p.dst[i];
    const uint4 *from = reinterpret_cast<const uint4 *>(codes + s * p.page_bytes);
    uint4 *to = reinterpret_cast<uint4 *>(codes + d * p.page_bytes);
    const int n = p.page_bytes / 16;
    constexpr int U = 8;
    int k = tid;
    for (; k + (U - 1) * COPY_THREADS < n; k += U * COPY_THREADS) {
        uint4 x[U];
#pragma unroll
        for (int j = 0; j < U; ++j) x[j] = __ldcs(from + k + j * COPY_THREADS);
#pragma unroll
        for (int j = 0; j < U; ++j) __stcs(to + k + j * COPY_THREADS, x[j]);
    }
    for (; k < n; k += COPY_THREADS) to[k] = from[k];
    for (int h = tid; h < p.c.hkv; h += COPY_THREADS) scales[d * p.c.hkv + h] = scales[s * p.c.hkv + h];
}

// Reordering of beams.  A beam's state is its table row; full pages are named
// by any number of rows, but the page being filled must be its row's own.  Of a
// parent's children one keeps that page (the parent itself, else the first) and
// each other one takes the page of a beam without children, of which there are
// exactly as many, and a copy of the tokens in it: nothing is allocated, and no
// page is both read and written.
constexpr int REORDER_BEAMS = 64, REORDER_THREADS = 256, REORDER_CTAS = 2432;

struct ReorderParams {
    CacheView c;
    const int *table, *lens, *parents;
    int *out;
    int beams, width;
};

// CTA (row, y): of the row's parts y, y + gridDim.y, ...: part 2 l + half is the
// copy, if it needs one, of K / V of layer l, the last one the table row.  Each
// CTA finds out by itself which rows copy (masks of children, two dependent
// loads), which is why it has several parts.  Measured: 64 beams in 36 layers of
// the 8B shape 40 us, of which K takes 14 (4 pieces of a thread in flight; with 8
// 47, a CTA a part 41); V's are pieces of 64-byte rows, whose 32-byte sectors the
// tokens fill in part.
template <int D, int P>
__global__ void __launch_bounds__(REORDER_THREADS) cache_reorder_kernel(const ReorderParams p) {
    __shared__ unsigned long long s_child[REORDER_BEAMS], s_extra, s_dead;
    const int tid = threadIdx.x, W = p.beams, row = blockIdx.x % W;
    const int64_t row0 = blockIdx.x - row;
    const int parts = 2 * p.c.layers + 1;
    const bool reports = row == 0 && (parts - 1) % gridDim.y == blockIdx.y;
    const int n = p.lens[row0];
    int parent = 0, wrong = 0;
    if (tid < W) {
        const int x = p.parents[row0 + tid], held = p.lens[row0 + tid];
        wrong = x < -1 || x >= W || held != n || n < 0 || (int64_t)n > (int64_t)p.width * P;
        if (wrong && reports) note_failure(p.c.status, MK_ERR_DEVICE_CHECK, (int)(row0 + tid), held, -1);
        parent = x == -1 ? tid : x;
    }
    if (tid < REORDER_BEAMS) s_child[tid] = 0;
    if (tid == 0) s_extra = s_dead = 0;
    const bool bad = __syncthreads_or(wrong);
    const int t = bad ? 0 : n / P, part = bad ? 0 : n % P;
    if (bad) parent = tid;  // each row stays as it is
    if (tid < W) atomicOr(&s_child[parent], 1ull << tid);
    __syncthreads();
    if (tid < W) {
        const unsigned long long children = s_child[parent];
        const int keeper = children >> parent & 1 ? parent : __ffsll((long long)children) - 1;
        if (keeper != tid) atomicOr(&s_extra, 1ull << tid);
        if (s_child[tid] == 0) atomicOr(&s_dead, 1ull << tid);
    }
    __syncthreads();
    int mine = 0;  // the row's parent
    while (!(s_child[mine] >> row & 1)) ++mine;
    int tail = mine;  // the row whose page being filled this one goes on with
    const bool copies = part && s_extra >> row & 1;
    if (copies) {
        unsigned long long dead = s_dead;
        for (int k = __popcll(s_extra & ((1ull << row) - 1)); k > 0; --k) dead &= dead - 1;
        tail = __ffsll((long long)dead) - 1;
    }
    const int *from = p.table + (row0 + mine) * p.width;
    int src = -1, dst = -1;
    if (part) {
        src = from[t];
        dst = p.table[(row0 + tail) * p.width + t];
    }
    const bool there = (unsigned)src < (unsigned)p.c.pages && (unsigned)dst < (unsigned)p.c.pages;
    for (int y = blockIdx.y; y < parts; y += gridDim.y) {
        if (y == parts - 1) {
            const int *self = p.table + (row0 + row) * p.width;
            for (int c = tid; c < p.width; c += REORDER_THREADS)
                p.out[(row0 + row) * p.width + c] = c < t ? from[c] : c == t && part ? dst : self[c];
            if (copies && !there && tid == 0)
                note_failure(p.c.status, MK_ERR_DEVICE_CHECK, (int)(row0 + row), t * P, (unsigned)src >= (unsigned)p.c.pages ? src : dst);
            continue;
        }
        if (!copies || !there || src == dst) continue;
        // The pages' 16-byte pieces of all heads, U of a thread in flight; those
        // behind the tokens are passed over.
        const bool values = y % 2;
        const size_t a = p.c.at(y / 2, src, 0), z = p.c.at(y / 2, dst, 0);
        uint8_t *codes = values ? p.c.v : p.c.k;
        float *scales = values ? p.c.vs : p.c.ks;
        const uint4 *in = reinterpret_cast<const uint4 *>(codes + a * P * D);
        uint4 *out = reinterpret_cast<uint4 *>(codes + z * P * D);
        constexpr int U = 4, PIECES = P * D / 16;
        const int all = p.c.hkv * PIECES;
        // bytes of piece i that hold tokens: K's token i / (D / 16); V's tokens 16 (i % (P / 16)) ..
        const auto bytes_of = [&](int i) {
            return values ? min(max(part - i % (P / 16) * 16, 0), 16) : i % PIECES / (D / 16) < part ? 16 : 0;
        };
        for (int i0 = tid; i0 < all; i0 += U * REORDER_THREADS) {
            uint4 x[U];
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int i = i0 + k * REORDER_THREADS;
                if (i < all && bytes_of(i)) x[k] = in[i];
            }
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int i = i0 + k * REORDER_THREADS;
                const int bytes = i < all ? bytes_of(i) : 0;
                if (bytes == 0) continue;
                if (bytes < 16) {  // the rest of these 16 stays: narrower stores (old bytes to mix in would have to be waited for)
                    uint8_t *to = reinterpret_cast<uint8_t *>(out + i);
                    uint32_t w = x[k].x;
                    if (bytes & 8) {
                        *reinterpret_cast<uint2 *>(to) = make_uint2(x[k].x, x[k].y);
                        w = x[k].z;
                        to += 8;
                    }
                    if (bytes & 4) {
                        *reinterpret_cast<uint32_t *>(to) = w;
                        w = bytes & 8 ? x[k].w : x[k].y;
                        to += 4;
                    }
                    if (bytes & 2) {
                        *reinterpret_cast<uint16_t *>(to) = (uint16_t)w;
                        w >>= 16;
                        to += 2;
                    }
                    if (bytes & 1) *to = (uint8_t)w;
                    continue;
                }
                out[i] = x[k];
            }
        }
        for (int h = tid; h < p.c.hkv; h += REORDER_THREADS) scales[z + h] = scales[a + h];
    }
}

static int move_params(const mk_cache_desc *cache, const mk_cache_rows *rows, const int32_t *table, int width,
                       const int32_t *start, const int32_t *count, int batch, int max_count, MoveParams &m) {
    if (int rc = cache_check(cache, m.c)) return rc;
    if (!rows || !rows->k || !rows->v || !table || !start || !count) return set_error(MK_ERR_INVALID, "null argument");
    if (batch < 0 || width <= 0 || max_count < 0 || rows->rows < 0)
        return set_error(MK_ERR_INVALID, "negative batch, count or rows, or an empty table");
    if (batch > 65535) return set_error(MK_ERR_UNSUPPORTED, "batch above 65535");
    if ((rows->k | rows->v) % 16) return set_error(MK_ERR_INVALID, "token rows must be 16-byte aligned");
    for (int i = 0; i < 4; ++i) {
        if (rows->k_stride[i] % 8 || rows->v_stride[i] % 8)
            return set_error(MK_ERR_INVALID, "token row strides must be multiples of 8 elements");
        m.r.ks[i] = rows->k_stride[i];
        m.r.vs[i] = rows->v_stride[i];
    }
    m.r.k = reinterpret_cast<uint16_t *>(rows->k);
    m.r.v = reinterpret_cast<uint16_t *>(rows->v);
    m.r.rows = rows->rows;
    m.r.row0 = reinterpret_cast<const int *>(rows->row0);
    m.table = table;
    m.start = start;
    m.count = count;
    m.width = width;
    m.max_count = std::min(max_count, rows->rows);
    return MK_OK;
}

using MoveFn = void (*)(const MoveParams);

static int launch_move(MoveFn f, const MoveParams &m, const mk_cache_desc *c, int batch, void *stream) {
    if (batch == 0 || m.max_count == 0) return MK_OK;
    const int P = c->page_tokens;
    const int64_t slots = std::min<int64_t>(((int64_t)m.max_count + 2 * P - 2) / P, m.width);
    if (slots * c->kv_heads > INT32_MAX) return set_error(MK_ERR_UNSUPPORTED, "too many pages in one call");
    f<<<dim3((unsigned)(slots * c->kv_heads), batch, c->layers), MOVE_THREADS, 0, static_cast<cudaStream_t>(stream)>>>(m);
    cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? MK_OK : serve_cuda_fail(e, "cache launch");
}

}  // namespace mk

using namespace mk;

extern "C" {

int mk_cache_store(const mk_cache_desc *cache, const mk_cache_rows *rows, const int32_t *table, int table_width,
                   const int32_t *start, const int32_t *count, int batch, int max_count, void *stream) {
    MoveParams m;
    if (int rc = move_params(cache, rows, table, table_width, start, count, batch, max_count, m)) return rc;
    const bool d64 = cache->head_dim == 64, p32 = cache->page_tokens == 32;
    if (m.max_count <= APPEND_TOKENS) {
        const int64_t heads = (int64_t)batch * cache->kv_heads, warps = heads * cache->layers;
        if (warps == 0 || m.max_count == 0) return MK_OK;
        if (heads > INT32_MAX || warps / (MOVE_THREADS / 32) >= INT32_MAX)
            return set_error(MK_ERR_UNSUPPORTED, "too many sequences and heads in one call");
        void (*g)(const MoveParams, int) = d64 ? (p32 ? cache_append_kernel<64, 32> : cache_append_kernel<64, 64>)
                                               : (p32 ? cache_append_kernel<128, 32> : cache_append_kernel<128, 64>);
        g<<<(unsigned)((warps + MOVE_THREADS / 32 - 1) / (MOVE_THREADS / 32)), MOVE_THREADS, 0,
            static_cast<cudaStream_t>(stream)>>>(m, (int)heads);
        cudaError_t e = cudaGetLastError();
        return e == cudaSuccess ? MK_OK : serve_cuda_fail(e, "cache append launch");
    }
    MoveFn f = d64 ? (p32 ? cache_store_kernel<64, 32> : cache_store_kernel<64, 64>)
                   : (p32 ? cache_store_kernel<128, 32> : cache_store_kernel<128, 64>);
    return launch_move(f, m, cache, batch, stream);
}

int mk_cache_load(const mk_cache_desc *cache, const mk_cache_rows *rows, const int32_t *table, int table_width,
                  const int32_t *start, const int32_t *count, int batch, int max_count, void *stream) {
    MoveParams m;
    if (int rc = move_params(cache, rows, table, table_width, start, count, batch, max_count, m)) return rc;
    const bool d64 = cache->head_dim == 64, p32 = cache->page_tokens == 32;
    MoveFn f = d64 ? (p32 ? cache_load_kernel<64, 32> : cache_load_kernel<64, 64>)
                   : (p32 ? cache_load_kernel<128, 32> : cache_load_kernel<128, 64>);
    return launch_move(f, m, cache, batch, stream);
}

int mk_cache_copy(const mk_cache_desc *cache, const int32_t *src, const int32_t *dst, int n, int32_t *table,
                  int64_t table_entries, void *stream) {
    CopyParams p;
    if (int rc = cache_check(cache, p.c)) return rc;
    if (n < 0 || (n > 0 && (!src || !dst)) || table_entries < 0 || (table_entries > 0 && !table))
        return set_error(MK_ERR_INVALID, "null page list or table, or a negative size");
    if (n == 0) return MK_OK;
    std::vector<uint8_t> role;
    std::vector<int> order;
    try {
        role.assign(cache->pages, 0);
        order.resize(n);
    } catch (const std::bad_alloc &) {
        return set_error(MK_ERR_INVALID, "out of host memory");
    }
    for (int i = 0; i < n; ++i) {
        if (src[i] < 0 || src[i] >= cache->pages || dst[i] < 0 || dst[i] >= cache->pages)
            return set_error(MK_ERR_INVALID, "page number out of range");
        if (role[dst[i]]) return set_error(MK_ERR_INVALID, "a destination page repeats, or is a source too");
        role[dst[i]] = 2;
        if (role[src[i]] == 2) return set_error(MK_ERR_INVALID, "a destination page repeats, or is a source too");
        role[src[i]] = 1;
        order[i] = i;
    }
    // by rising src (the first listed first): one launch renames with a binary
    // search, and a src whose copies span two launches is renamed by the first,
    // after which no entry names it
    std::sort(order.begin(), order.end(), [&](int a, int b) { return src[a] != src[b] ? src[a] < src[b] : a < b; });
    p.page_bytes = cache->kv_heads * cache->page_tokens * cache->head_dim;
    p.table = table;
    p.entries = table ? table_entries : 0;
    for (int at = 0; at < n; at += COPY_PAIRS) {
        p.n = std::min(COPY_PAIRS, n - at);
        for (int i = 0; i < p.n; ++i) {
            p.src[i] = src[order[at + i]];
            p.dst[i] = dst[order[at + i]];
        }
        const unsigned y = 2u * cache->layers + (p.entries ? 1 : 0);
        if (y > 65535) return set_error(MK_ERR_UNSUPPORTED, "too many layers");
        cache_copy_kernel<<<dim3(p.n, y), COPY_THREADS, 0, static_cast<cudaStream_t>(stream)>>>(p);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return serve_cuda_fail(e, "page copy launch");
    }
    return MK_OK;
}

int mk_cache_reorder(const mk_cache_desc *cache, const int32_t *table, const int32_t *lens, const int32_t *parents,
                     int32_t *table_out, int batch, int beams, int table_width, void *stream) {
    ReorderParams p;
    if (int rc = cache_check(cache, p.c)) return rc;
    if (batch < 0 || beams <= 0 || table_width <= 0) return set_error(MK_ERR_INVALID, "negative batch, no beams or an empty table");
    if (beams > REORDER_BEAMS) return set_error(MK_ERR_UNSUPPORTED, "more than 64 beams");
    const int64_t rows = (int64_t)batch * beams;
    if (rows > INT32_MAX || 2 * cache->layers + 1 > 65535) return set_error(MK_ERR_UNSUPPORTED, "too many rows or layers");
    if (rows == 0) return MK_OK;
    if (!table || !lens || !parents || !table_out) return set_error(MK_ERR_INVALID, "null argument");
    if (table < table_out + rows * table_width && table_out < table + rows * table_width)
        return set_error(MK_ERR_INVALID, "the new table overlaps the old one");
    p.table = table;
    p.lens = lens;
    p.parents = parents;
    p.out = table_out;
    p.beams = beams;
    p.width = table_width;
    const bool p32 = cache->page_tokens == 32;
    void (*f)(const ReorderParams) = cache->head_dim == 64 ? (p32 ? cache_reorder_kernel<64, 32> : cache_reorder_kernel<64, 64>)
                                                           : (p32 ? cache_reorder_kernel<128, 32> : cache_reorder_kernel<128, 64>);
    const int64_t each = std::max<int64_t>(1, std::min<int64_t>(2 * cache->layers + 1, (REORDER_CTAS + rows - 1) / rows));
    f<<<dim3((unsigned)rows, (unsigned)each), REORDER_THREADS, 0, static_cast<cudaStream_t>(stream)>>>(p);
    cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? MK_OK : serve_cuda_fail(e, "reorder launch");
}

int mk_cache_status(const mk_cache_desc *cache, int clear, int32_t *status, void *stream) {
    CacheView v;
    if (int rc = cache_check(cache, v)) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int32_t w[4];
    cudaError_t e = cudaMemcpyAsync(w, v.status, sizeof w, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess && clear) e = cudaMemsetAsync(v.status, 0, sizeof w, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e != cudaSuccess) return serve_cuda_fail(e, "read cache status");
    if (status) std::memcpy(status, w, sizeof w);
    if (!w[0]) return MK_OK;
    return set_error(w[0], "cache check failed: sequence " + std::to_string(w[1]) + " position " + std::to_string(w[2]) +
                               " page " + std::to_string(w[3]));
}

}  // extern "C"
