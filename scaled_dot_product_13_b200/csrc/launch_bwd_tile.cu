// Launch unit of the warp-tile backward kernel.
#include "bwd_tile.cuh"
#include "launch_bwd.h"

namespace sdpa {

namespace {

template <bool kBF16>
sdpa_status run(const BwdLaunch &ln, std::string *err) {
  const Problem &pb = ln.pb;
  auto kern = bwd_tile_kernel<kBF16>;
  // the limit for the largest head dims, set once
  sdpa_status st = prepare_kernel((const void *)kern, kBwdTileThreads, bwd_tile_smem(512, 512),
                                  "bwd_tile_kernel", err);
  if (st != SDPA_OK) return st;
  BwdParams p;
  fill_bwd_params(ln, &p);
  auto parts = [](int d) { return (d + kBwdTileCols - 1) / kBwdTileCols; };
  const long long slabs = (long long)pb.B * pb.Hkv;
  BwdTileGrid g;
  g.key_tiles = (pb.S + kBwdTileX - 1) / kBwdTileX;
  g.key_parts = parts(pb.Dqk > pb.Dv ? pb.Dqk : pb.Dv);
  g.row_tiles = (p.a.R + kBwdTileX - 1) / kBwdTileX;
  g.row_parts = parts(pb.Dqk);
  g.key_ctas = slabs * g.key_tiles * g.key_parts;
  const long long ctas = g.key_ctas + slabs * g.row_tiles * g.row_parts;
  if (ctas > 0x7fffffffLL) {
    *err = "problem needs more than 2^31 CTAs";
    return SDPA_ERR_UNSUPPORTED;
  }
  kern<<<(unsigned)ctas, kBwdTileThreads, bwd_tile_smem(pb.Dqk, pb.Dv), ln.stream>>>(p, g);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    *err = std::string("bwd_tile_kernel launch failed: ") + cudaGetErrorString(e);
    return SDPA_ERR_CUDA;
  }
  return SDPA_OK;
}

}  // namespace

sdpa_status launch_bwd_tile(const BwdLaunch &ln, std::string *err) {
  return ln.pb.dtype == SDPA_BF16 ? run<true>(ln, err) : run<false>(ln, err);
}

}  // namespace sdpa
