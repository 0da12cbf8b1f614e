// gated_geo.hpp -- where the threads of a gated scan's tile read and write.
// It follows fused_common.hpp, whose tile geometry it starts from; apart from
// the rest of the kernels, so that it can be checked on the host.
#pragma once

namespace lrscan {

namespace {

// How rows lie.  kWhole: at least one vector long, but not made of aligned
// vectors.  Its last, partial vector is moved back to start at D - V, so that
// every access is one of 16 bytes; the columns it shares with its neighbour
// are computed twice, to the same bits.  (With the partial vector tested for at
// every access instead, fp32 [5, 777, 1023] took 28.8 us forward and 46.5
// reverse, against 19.2 and 33.3 for rows of 1024.)  kNarrow: shorter than a
// vector, element by element.
enum RowKind { kAligned, kWhole, kNarrow };

template <class C, int RK, bool REV>
__device__ __forceinline__ Geo gated_geo(uint32_t ticket, const Dims& d, int wave, int rg, int cg) {
    Geo g = tile_geo<C, REV>(ticket, d, wave, rg, cg);
    if constexpr (RK == kWhole) {
        // bases are taken 16 bytes before the tile, so that offsets stay positive
        g.tbase -= 16;
        g.coff += 16;
        if (g.nvalid < C::V) {
            // threads past the row read this vector too: a tile's first column
            // may have fewer than V after it
            g.coff = (uint32_t)((d.D - C::V - g.dcol0) * C::EB + 16);
            if (g.nvalid > 0) {
                g.d0 = d.D - C::V;
                g.nvalid = C::V;
            }
        }
    }
    return g;
}

// The column of a tile's slot c (D or more: none).
template <class C, int RK>
__device__ __forceinline__ int slot_column(const Geo& g, int c, int D) {
    const int d0 = g.dcol0 + c / C::V * C::V;
    return (RK == kWhole && d0 < D && d0 + C::V > D ? D - C::V : d0) + c % C::V;
}

}  // namespace

}  // namespace lrscan
