// Tensors of several strided dimensions as the entry points check them (internal to the library).
#pragma once

#include "work.hpp"

#include <initializer_list>

namespace {

// A tensor of up to three strided dimensions over rows of `width` elements.
struct Dim {
    uint64_t extent, stride;
};

struct Grid {
    const void* p = nullptr;
    Dim given[3] = {{1, 0}, {1, 0}, {1, 0}};   // as the caller names them
    Dim dim[3] = {{1, 0}, {1, 0}, {1, 0}};     // by ascending stride, those of one element left out
    int dims = 0;
    uint64_t width = 0, size = 0;
    bool empty = true;

    Grid() = default;
    Grid(const void* at, uint64_t w, uint64_t elem, std::initializer_list<Dim> ds) : p(at), width(w), size(elem), empty(at == nullptr || w == 0) {
        int n = 0;
        for (const Dim& d : ds) {
            given[n++] = d;
            if (d.extent == 0) empty = true;
            if (d.extent > 1) dim[dims++] = d;
        }
        std::sort(dim, dim + dims, [](const Dim& x, const Dim& y) { return x.stride < y.stride; });
    }
    // No two of its rows share an element, as far as nested dimensions show it.  (Strides below
    // 2^40 and a span below 2^56, as check_grid has them.)
    bool apart() const {
        uint64_t span = width;
        for (int i = 0; i < dims; ++i) {
            if (dim[i].stride < span) return false;
            span += dim[i].stride * (dim[i].extent - 1);
        }
        return true;
    }
    bool in_range() const {
        unsigned __int128 s = width;
        for (int i = 0; i < dims; ++i) {
            if (dim[i].stride >> 40) return false;
            s += static_cast<unsigned __int128>(dim[i].stride) * (dim[i].extent - 1);
        }
        return s >> 56 == 0;
    }
    uint64_t span() const {
        uint64_t s = width;
        for (int i = 0; i < dims; ++i) s += dim[i].stride * (dim[i].extent - 1);
        return s;
    }
    // As rows an equal distance apart where it is that; else its span.
    Extent extent() const {
        if (empty) return {nullptr, 0, 0, 0, size};
        uint64_t w = width;
        int i = 0;
        while (i < dims && dim[i].stride == w) w *= dim[i++].extent;
        if (i == dims) return {p, 1, w, w, size};
        Dim rows = dim[i];
        for (++i; i < dims && dim[i].stride == rows.stride * rows.extent; ++i) rows.extent *= dim[i].extent;
        if (i == dims && rows.stride >= w) return {p, rows.extent, w, rows.stride, size};
        return {p, 1, span(), span(), size};
    }
    // Every element where the other has it: the strides are compared dimension by dimension, but for
    // those of one element.  (Sorted ones would take a transposition of equal extents for the same.)
    bool same(const Grid& o) const {
        if (p != o.p || width != o.width || size != o.size) return false;
        for (int i = 0; i < 3; ++i)
            if (given[i].extent != o.given[i].extent || (given[i].extent > 1 && given[i].stride != o.given[i].stride)) return false;
        return true;
    }
};

fa_status check_grid(fa_work* w, const Grid& g, const char* name) {
    if (g.empty && g.p) return FA_OK;              // nothing of it is read
    if (!g.in_range()) return fail(w, FA_ERR_RANGE, std::string(name) + ": a stride of 2^40 or more, or a span of 2^56");
    if (reinterpret_cast<uintptr_t>(g.p) % g.size) return fail(w, FA_ERR_ARG, std::string(name) + " is not aligned to its element type");
    return check_ptr(w, g.p, name);
}

fa_status check_out(fa_work* w, const Grid& g, const char* name) {
    const fa_status r = check_grid(w, g, name);
    if (r != FA_OK || g.empty || g.apart()) return r;
    return fail(w, FA_ERR_RANGE, std::string(name) + ": strides by which its rows overlap");
}

}  // namespace
