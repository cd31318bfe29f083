// tile_order.h for the host, behind a C interface (tests/test_tile_order.py).
#include "tile_order.h"

extern "C" int remap(int i, int n) { return tre::xcd_remap(i, n); }
extern "C" int remap_rounds8(int i, int n) { return tre::xcd_remap_rounds<8>(i, n); }
extern "C" int remap_rounds32(int i, int n) { return tre::xcd_remap_rounds<32>(i, n); }
extern "C" int uneven(const int32_t* offs, int E) { return tre::uneven_eighths(offs, E); }
