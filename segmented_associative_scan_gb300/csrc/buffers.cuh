// What the C entry points of the sequence-model operators and of the losses share: the checks of
// a call's buffers, and launches by data type.
#pragma once

#include <cstdint>
#include <type_traits>

#include "../../include/rlca.h"
#include "sequence.cuh"

namespace rlca {
namespace seq {

inline size_t bytes_of(Fmt f) { return f == Fmt::kF32 ? 4 : 2; }

constexpr int64_t kMaxExtent = INT64_C(1) << 60;  // bytes any array may span

// The bytes an array spans, and how its elements lie in them: `width` bytes at every
// multiple of `unit` (the smaller stride) when `regular`.
struct Extent {
    const void *ptr = nullptr;
    uintptr_t lo = 0, hi = 0;
    bool regular = false;
    uintptr_t unit = 0, width = 0;
};

inline bool overlaps(const Extent &a, const Extent &b)
{
    if (a.lo >= a.hi || b.lo >= b.hi || a.lo >= b.hi || b.lo >= a.hi) return false;
    if (a.regular && b.regular && a.unit == b.unit) {
        // Side by side within every stride.
        const uintptr_t d = (b.lo >= a.lo ? b.lo - a.lo : a.unit - (a.lo - b.lo) % a.unit) % a.unit;
        if (d >= a.width && d + b.width <= a.unit) return false;
    }
    return true;
}

// Collects a call's buffers and answers for all of them at once; the first failed check of
// each kind wins in the order shape, null, alias, memory.
class Buffers {
public:
    Buffers(int64_t N, int64_t T) : N_(N), T_(T) {}

    void in(const void *p, int64_t count, size_t elem, bool required = true)
    {
        flat(p, count, elem, required, false);
    }
    void out(const void *p, int64_t count, size_t elem, bool required = true)
    {
        flat(p, count, elem, required, true);
    }
    // A state and its new value, which may be exactly the state (updated in place): that pair
    // overlaps, and no other may.
    void state(const void *p, const void *new_state, int64_t count, size_t elem, bool required)
    {
        if (count > 0 && p && p == new_state) {
            state_in_ = n_in_;
            state_out_ = n_out_;
        }
        flat(p, count, elem, required, false);
        flat(new_state, count, elem, true, true);
    }
    // A boundary that the kernels' accesses of several elements need.
    void aligned(const void *p, size_t bytes)
    {
        misaligned_ |= reinterpret_cast<uintptr_t>(p) % bytes != 0;
    }
    // An input of one value per step: N rows of T, any distance apart.
    void line(const void *p, int64_t ld, size_t elem, bool required)
    {
        if (N_ <= 0 || T_ <= 0) return;
        if (!p) {
            null_ |= required;
            return;
        }
        if (ld < 0 || (__int128)N_ * ld > kMaxExtent) {
            shape_ = true;
            return;
        }
        in(p, (N_ > 1 ? (N_ - 1) * ld : 0) + T_, elem);
    }
    // An activation and a result in its layout, which may be exactly that activation (written in
    // place): that pair overlaps, and no other may.
    void in_place(const rlca_steps &a, const rlca_steps &result, int64_t width, size_t elem)
    {
        const int in = n_in_, out = n_out_;
        steps(a, width, elem, true, false);
        steps(result, width, elem, true, true);
        if (n_in_ > in && n_out_ > out && a.ptr == result.ptr &&
            (N_ <= 1 || a.row == result.row) && (T_ <= 1 || a.step == result.step)) {
            state_in_ = in;
            state_out_ = out;
        }
    }
    void steps(const rlca_steps &a, int64_t width, size_t elem, bool required, bool output)
    {
        if (N_ <= 0 || T_ <= 0 || width <= 0) return;
        if (!a.ptr) {
            null_ |= required;
            return;
        }
        const int64_t row = N_ > 1 ? a.row : 0, step = T_ > 1 ? a.step : 0;
        if (row < 0 || step < 0) {
            shape_ = true;
            return;
        }
        const __int128 span = ((__int128)(N_ - 1) * row + (__int128)(T_ - 1) * step + width) *
                              (__int128)elem;
        if (span > kMaxExtent) {
            shape_ = true;
            return;
        }
        // Nested strides: the inner one holds a row of channels, the outer all of the inner.
        const bool by_step = N_ == 1 || (T_ > 1 && step <= row);
        const int64_t inner = by_step ? step : row, outer = by_step ? row : step;
        const int64_t n_in = by_step ? T_ : N_, n_out = by_step ? N_ : T_;
        const bool nested = (n_in == 1 || inner >= width) &&
                            (n_out == 1 || outer >= inner * (n_in - 1) + width);
        if (output && !nested) {
            shape_ = true;
            return;
        }
        Extent e;
        e.ptr = a.ptr;
        e.lo = reinterpret_cast<uintptr_t>(a.ptr);
        misaligned_ |= e.lo % elem != 0;
        e.hi = e.lo + (uintptr_t)span;
        const int64_t unit = n_in > 1 ? inner : outer;
        if (nested && unit > 0 && (n_in == 1 || n_out == 1 || outer % inner == 0)) {
            e.regular = true;
            e.unit = (uintptr_t)unit * elem;
            e.width = (uintptr_t)width * elem;
        }
        add(e, output);
    }
    void rows(const rlca_rows &r)
    {
        if (N_ <= 0) return;
        if (T_ > 0 && (r.terminated || r.truncated)) {
            if (r.flag_ld < T_ || (__int128)N_ * r.flag_ld > kMaxExtent) {
                shape_ = true;
                return;
            }
            const int64_t n = (N_ - 1) * r.flag_ld + T_;
            in(r.terminated, n, 1, false);
            in(r.truncated, n, 1, false);
        }
        in(r.lengths, N_, 4, false);
    }

    int check(void *ws, size_t ws_bytes, size_t need) const
    {
        if (shape_ || over_) return RLCA_ERR_SHAPE;
        if (null_) return RLCA_ERR_NULL;
        for (int i = 0; i < n_out_; ++i) {
            for (int k = 0; k < n_in_; ++k)
                if (overlaps(out_[i], in_[k]) && !(i == state_out_ && k == state_in_))
                    return RLCA_ERR_ALIAS;
            for (int k = i + 1; k < n_out_; ++k)
                if (overlaps(out_[i], out_[k])) return RLCA_ERR_ALIAS;
        }
        if (need) {
            if (!ws || ws_bytes < need || reinterpret_cast<uintptr_t>(ws) % 256)
                return RLCA_ERR_WORKSPACE;
            Extent w;
            w.ptr = ws;
            w.lo = reinterpret_cast<uintptr_t>(ws);
            w.hi = w.lo + need;
            for (int k = 0; k < n_in_; ++k)
                if (overlaps(w, in_[k])) return RLCA_ERR_ALIAS;
            for (int k = 0; k < n_out_; ++k)
                if (overlaps(w, out_[k])) return RLCA_ERR_ALIAS;
        }
        if (misaligned_) return RLCA_ERR_MEMORY;
        // Checked last, as it asks the CUDA runtime.
        int device = 0;
        if (cudaGetDevice(&device) != cudaSuccess) {
            (void)cudaGetLastError();
            return RLCA_ERR_LAUNCH;
        }
        for (int k = 0; k < n_in_; ++k)
            if (!reachable(in_[k].ptr, device)) return RLCA_ERR_MEMORY;
        for (int k = 0; k < n_out_; ++k)
            if (!reachable(out_[k].ptr, device)) return RLCA_ERR_MEMORY;
        if (need && !reachable(ws, device)) return RLCA_ERR_MEMORY;
        return RLCA_OK;
    }

private:
    static bool reachable(const void *ptr, int device)
    {
        cudaPointerAttributes a;
        if (cudaPointerGetAttributes(&a, ptr) != cudaSuccess) {
            (void)cudaGetLastError();
            return false;
        }
        return a.type == cudaMemoryTypeManaged ||
               (a.type == cudaMemoryTypeDevice && a.device == device);
    }
    void flat(const void *p, int64_t count, size_t elem, bool required, bool output)
    {
        if (count <= 0) return;
        if (!p) {
            null_ |= required;
            return;
        }
        Extent e;
        e.ptr = p;
        e.lo = reinterpret_cast<uintptr_t>(p);
        misaligned_ |= e.lo % elem != 0;
        e.hi = e.lo + (uintptr_t)count * elem;
        add(e, output);
    }
    void add(const Extent &e, bool output)
    {
        if (output ? n_out_ == kMax : n_in_ == kMax)
            over_ = true;
        else if (output)
            out_[n_out_++] = e;
        else
            in_[n_in_++] = e;
    }

    static constexpr int kMax = 16;
    int64_t N_, T_;
    Extent in_[kMax], out_[kMax];
    int n_in_ = 0, n_out_ = 0;
    int state_in_ = -1, state_out_ = -1;
    bool shape_ = false, null_ = false, over_ = false, misaligned_ = false;
};

inline bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Every row of every step starts on a 16-byte boundary.
inline bool vectors(const rlca_steps &a, int64_t N, int64_t T, int V)
{
    return !a.ptr ||
           (aligned16(a.ptr) && (N <= 1 || a.row % V == 0) && (T <= 1 || a.step % V == 0));
}

inline int status(cudaError_t e)
{
    if (e == cudaSuccess) return RLCA_OK;
    (void)cudaGetLastError();
    return RLCA_ERR_LAUNCH;
}

template <typename Launch>
cudaError_t in_format(Fmt f, Launch launch)
{
    switch (f) {
    case Fmt::kF32: return launch(std::integral_constant<Fmt, Fmt::kF32>{});
    case Fmt::kBF16: return launch(std::integral_constant<Fmt, Fmt::kBF16>{});
    default: return launch(std::integral_constant<Fmt, Fmt::kF16>{});
    }
}

inline bool product_fits(int64_t a, int64_t b, int64_t c, int64_t d)
{
    return (__int128)a * b < kMaxExtent && (__int128)a * b * c < kMaxExtent &&
           (__int128)a * b * c * d < kMaxExtent;
}

}  // namespace seq
}  // namespace rlca
