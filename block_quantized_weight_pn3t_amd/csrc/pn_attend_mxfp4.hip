// pn_attend_mxfp4.hip -- the attention kernels over MXFP4 caches.
#include "pn_attend.h"

namespace pn {
PN_ATTEND_FORMAT(PN_CACHE_MXFP4)
}  // namespace pn
